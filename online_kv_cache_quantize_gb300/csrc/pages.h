// Parameter blocks and launchers of the page calls (internal; pages.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace tqk {

constexpr int kSegPages = 4096;               // pages per segment of the free-page index
constexpr int kSegWords = kSegPages / 32;
constexpr int kMaxSegs = 4096;                // so at most 2^24 pages
constexpr int kMaxPageTables = 4;             // tables one compaction rewrites
constexpr int kPagePlanes = 6;
// Calls of more rows than this add up the rows before a row by blocks of
// kRowBlock (one launch more, and two for a fork's parents), so that their work
// grows with the rows and not with their square: trim and reserve of 65536 rows
// 615 -> 435 us, trim and fork 1735 -> 612 us. The launches cost 1 and 3 us, which
// the sums over all rows save from about 4096 rows on (fork 44.0 -> 42.8 us).
constexpr int kManyRows = 2048;
constexpr int kRowBlock = 256;

// A pool as the kernels see it: page p of plane q is units[q] consecutive
// 16-byte units from unit p * units[q] of base[q]; the planes of a page
// follow one another as units [off[q], off[q + 1]) of it.
struct PoolParams {
    char* base[kPagePlanes];
    int units[kPagePlanes];
    int off[kPagePlanes + 1];
    int32_t* refs;
    int n_pages;
    int page;   // tokens
    int slots;  // of a page: tokens x KV heads
};

struct TableParams {
    int32_t* e;
    int64_t stride;
    int rows, max_pages;
};

// The free-page index of a pool, formed by the first launch of a call from
// the counts as they stood: a bit per page (set: free), per 32-page word the
// free pages of its segment before it, per segment its free pages.
struct PageIndex {
    uint32_t* bits;    // [segs * kSegWords]
    uint16_t* before;  // [segs * kSegWords]
    int32_t* count;    // [segs]
    int segs;
};

struct ReserveParams {
    PoolParams pool;
    PageIndex ix;
    TableParams t;
    const int32_t* lengths;
    const int32_t* add;  // NULL: add_all for every row
    int add_all;
    int32_t* blocks;     // [rows / kRowBlock] requests of a block of rows, NULL up to kManyRows rows
    int32_t* need;       // [rows] twice a row's requests, + 1 where the first is for a copy of its last page
    int32_t* shortage;   // may be NULL
    int32_t* granted;    // [rows], may be NULL
    __device__ int rows() const { return t.rows; }
    __device__ int asks(int row) const { return need[row] >> 1; }
};

struct ForkParams {
    PoolParams pool;
    PageIndex ix;
    TableParams src, dst;
    const int32_t* parent;
    const int32_t* src_lengths;
    int32_t* dst_lengths;  // may be NULL
    int keep_src;
    int32_t* tail;         // [dst.rows] page to copy for the row, or -1
    int32_t* blocks;       // [dst.rows / kRowBlock] copies of a block of rows; this and the next two NULL up to kManyRows rows
    int32_t* first;        // [src.rows] first child of a row
    int32_t* children;     // [src.rows] how many it has
    int32_t* shortage;     // may be NULL
    int chunks;            // CTAs per page copied
    __device__ int rows() const { return dst.rows; }
    __device__ int asks(int row) const { return tail[row] >= 0 ? 1 : 0; }
};

struct TrimParams {
    PoolParams pool;
    TableParams t;
    const int32_t* lengths;
    int window, sinks;
};

struct CopyParams {
    PoolParams src, dst;
    const int32_t* from;
    const int32_t* to;
    int n, chunks;
    int ctas;
    uint32_t* err;  // device error word
};

struct CompactParams {
    PoolParams src, dst;
    PageIndex ix;
    TableParams from[kMaxPageTables], to[kMaxPageTables];
    int n_tables;
    int in_place;
    int2* move;       // [n_pages] (page, new page)
    int32_t* map;     // [n_pages] new page, or -1
    int32_t* n_move;  // [1]
    int32_t* live;    // may be NULL
    int chunks;
    int ctas;       // of the launch that moves
    uint32_t* err;  // device error word
};

cudaError_t launch_pages_reserve(const ReserveParams& p, cudaStream_t s);
cudaError_t launch_pages_fork(const ForkParams& p, cudaStream_t s);
cudaError_t launch_pages_trim(const TrimParams& p, cudaStream_t s);
cudaError_t launch_pages_copy(const CopyParams& p, cudaStream_t s);
cudaError_t launch_pages_compact(const CompactParams& p, cudaStream_t s);

// CTAs that copy one page of `units` 16-byte units
int page_copy_chunks(int units);

}  // namespace tqk
