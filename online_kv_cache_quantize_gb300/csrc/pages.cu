// Pages of a packed cache: reserving, forking, giving back, copying and
// compacting them, with all bookkeeping on the device (a serving loop that
// forks, grows and trims its sequences needs no host round trip and can be
// captured in a graph).
//
// State. refs[p] counts the table entries that hold page p; 0 is free. There
// is no free list: "the r-th request takes the r-th lowest free page", so a
// call's result follows from its inputs alone, whatever order its CTAs run in,
// and nothing besides the counts can fall out of step with the tables.
//
// The r-th lowest free page comes from a two-level index (bits and prefix
// counts per 4096-page segment) that the first launch of a call builds in one
// pass over the counts, one CTA per segment; the second launch's CTAs add up
// the segments' counts and find their pages by themselves, in parallel.
// What bounds these calls is latency (two dependent launches, a few L2 round
// trips in each) until the copied pages outweigh it. A fork copies its few pages
// through registers (16 bytes per thread and load, eight loads in flight), where
// a copy starts soonest; the calls that move many pages are bound by HBM and
// stream them through shared memory with bulk copies (stream_pages). Measured in a
// graph: trim and reserve of 256 rows of a pool of 65 K pages 10.4 us; a fork of 16
// rows into 128, a 104 KB copy each, 14.4 us (27 MB, 4 us at the copy rate); a
// compaction of 1552 pages of 52 KB 35.9 us (162 MB, 23.9 us), 10 us of it the
// index and the map.
#include "common.cuh"
#include "pages.h"
#include "pipeline.cuh"

namespace tqk {

namespace {

constexpr int kPageThreads = 256;
constexpr int kCopyPer = 8;                                // 16-byte units a thread has in flight
constexpr int kCopyUnits = kPageThreads * kCopyPer;        // 32 KB per CTA

__device__ __forceinline__ void wait_prior_grid() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void let_next_grid() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// A call's first launch is a programmatic dependent too, of whatever is before it
// on the stream: it waits for that, and only then lets its own dependent start,
// so that nothing of the call runs before what came before it is complete.
__device__ __forceinline__ void begin_call() {
    wait_prior_grid();
    let_next_grid();
}

__device__ __forceinline__ bool page_ok(int p, int n) { return (unsigned)p < (unsigned)n; }

// exclusive prefix sum over the CTA's kPageThreads threads; *total = the sum
__device__ __forceinline__ int block_prefix(int v, int* total) {
    __shared__ int s_w[kPageThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(TQ_FULL_MASK, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // s_w may still be read by an earlier call
    if (lane == 31) s_w[warp] = x;
    __syncthreads();
    int base = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kPageThreads / 32; ++w) {
        if (w < warp) base += s_w[w];
        sum += s_w[w];
    }
    *total = sum;
    return base + x - v;
}

__device__ __forceinline__ int block_sum(int v) {
    int total;
    block_prefix(v, &total);
    return total;
}

// Segment `seg` of the index: word w = pages seg * 4096 + 32 w .. + 31.
__device__ __forceinline__ void index_segment(const PoolParams& pool, const PageIndex& ix, int seg) {
    constexpr int kWarps = kPageThreads / 32, kPer = kSegWords / kWarps;
    __shared__ uint32_t s_bits[kSegWords];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int r[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int64_t p = (int64_t)seg * kSegPages + (warp * kPer + k) * 32 + lane;
        r[k] = p < pool.n_pages ? pool.refs[p] : 1;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const uint32_t b = __ballot_sync(TQ_FULL_MASK, r[k] <= 0);
        if (lane == 0) s_bits[warp * kPer + k] = b;
    }
    __syncthreads();
    const int w = threadIdx.x;
    const uint32_t b = w < kSegWords ? s_bits[w] : 0u;
    int total;
    const int before = block_prefix(__popc(b), &total);
    if (w < kSegWords) {
        ix.bits[(int64_t)seg * kSegWords + w] = b;
        ix.before[(int64_t)seg * kSegWords + w] = (uint16_t)before;
    }
    if (w == 0) ix.count[seg] = total;
}

// the (n + 1)-th set bit of w
__device__ __forceinline__ int nth_bit(uint32_t w, int n) {
    for (int i = 0; i < n; ++i) w &= w - 1u;
    return __ffs(w) - 1;
}

// Exclusive prefix of the segments' free pages into shared memory, s_pre[segs]
// = all of them. Called by the whole CTA.
__device__ __forceinline__ void load_prefix(const PageIndex& ix, int* s_pre) {
    int base = 0;
    for (int s0 = 0; s0 < ix.segs; s0 += kPageThreads) {
        const int s = s0 + threadIdx.x;
        int total;
        const int pre = block_prefix(s < ix.segs ? ix.count[s] : 0, &total);
        if (s < ix.segs) s_pre[s] = base + pre;
        base += total;
    }
    if (threadIdx.x == 0) s_pre[ix.segs] = base;
    __syncthreads();
}

// Sum of f over the rows before `row`, in parallel over the CTA; `blocks` (may
// be NULL) holds the sums of whole blocks of rows.
template <typename F>
__device__ __forceinline__ int rows_before(int row, const int32_t* blocks, F f) {
    const int whole = blocks ? row / kRowBlock : 0;
    int sum = 0;
    for (int b = threadIdx.x; b < whole; b += kPageThreads) sum += blocks[b];
    for (int r = whole * kRowBlock + (int)threadIdx.x; r < row; r += kPageThreads) sum += f(r);
    return block_sum(sum);
}

// The r-th lowest free page (from 0), r below the number of free pages; one
// thread, the prefix in shared memory.
__device__ __forceinline__ int find_free(const PageIndex& ix, const int* s_pre, int r) {
    int lo = 0, hi = ix.segs;  // s_pre[lo] <= r < s_pre[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (s_pre[m] <= r) lo = m;
        else hi = m;
    }
    const int q = r - s_pre[lo];
    const uint16_t* before = ix.before + (int64_t)lo * kSegWords;
    int a = 0, b = kSegWords;  // before[a] <= q, and q < before[b] where b < kSegWords
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        const int m = (a + b) >> 1;
        if (before[m] <= q) a = m;
        else b = m;
    }
    return lo * kSegPages + a * 32 + nth_bit(ix.bits[(int64_t)lo * kSegWords + a], q - before[a]);
}

// free pages below page p (p <= n_pages)
__device__ __forceinline__ int free_below(const PageIndex& ix, const int* s_pre, int p) {
    const int seg = p / kSegPages;
    if (seg >= ix.segs) return s_pre[ix.segs];
    const int w = (p % kSegPages) >> 5;
    const int64_t i = (int64_t)seg * kSegWords + w;
    return s_pre[seg] + ix.before[i] + __popc(ix.bits[i] & ((1u << (p & 31)) - 1u));
}

// 32 KB of page `from` of one pool into page `to` of another (chunk c of it)
__device__ __forceinline__ void copy_chunk(const PoolParams& src, const PoolParams& dst, int64_t from, int64_t to, int c) {
    const int total = src.off[kPagePlanes];
    const int u0 = c * kCopyUnits + (int)threadIdx.x;
    uint4 v[kCopyPer];
    char* out[kCopyPer];
#pragma unroll
    for (int k = 0; k < kCopyPer; ++k) {
        const int u = u0 + k * kPageThreads;
        out[k] = nullptr;
        if (u < total) {
            const char* b = src.base[0];
            char* o = dst.base[0];
            int n = src.units[0], rel = u;
#pragma unroll
            for (int q = 1; q < kPagePlanes; ++q)
                if (u >= src.off[q]) {
                    b = src.base[q];
                    o = dst.base[q];
                    n = src.units[q];
                    rel = u - src.off[q];
                }
            v[k] = *reinterpret_cast<const uint4*>(b + (from * n + rel) * 16);
            out[k] = o + (to * n + rel) * 16;
        }
    }
#pragma unroll
    for (int k = 0; k < kCopyPer; ++k)
        if (out[k]) *reinterpret_cast<uint4*>(out[k]) = v[k];
}

// Streams pieces of pages through a ring in shared memory: one warp of each of
// `ctas` CTAs takes the pieces blockIdx.x, blockIdx.x + ctas, ... of `work`
// (page i / chunks of the list that `at` reads as (from, to), piece i % chunks),
// loads kLag of them ahead and stores each as it lands; lane q < 6 issues the
// part of a piece that lies in plane q. No register carries data, and 128 KB per
// SM are in flight. Compacting 1552 pages of 52 KB took 63.6 us with 16-byte
// loads and stores, 51.3 us with one thread issuing all parts (2 us a piece, all
// of it address arithmetic) and 35.6 us so.
constexpr int kRing = 6;
constexpr int kLag = kRing - 2;  // pieces between a load and its store
constexpr size_t kRingBytes = (size_t)kRing * kCopyUnits * 16;

template <typename At>
__device__ __forceinline__ void stream_pages(const PoolParams& src, const PoolParams& dst, At at, int64_t work, int chunks,
                                             int ctas, uint32_t* err) {
    extern __shared__ __align__(128) unsigned char ring_smem[];
    __shared__ __align__(8) uint64_t s_bar[kRing];
    const uint32_t bar0 = (uint32_t)__cvta_generic_to_shared(s_bar), ring = (uint32_t)__cvta_generic_to_shared(ring_smem);
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(bar0 + 8 * i, 1);
        mbar_init_fence();
    }
    __syncwarp();
    // pieces of one size: CTAs take every ctas-th piece, which can be the same
    // one of each page
    const int total = src.off[kPagePlanes], size = (total + chunks - 1) / chunks;
    // this lane's plane: units [o0, o1) of a page
    const char* in = nullptr;
    char* out = nullptr;
    int64_t stride = 0;
    int o0 = 0, o1 = 0;
#pragma unroll
    for (int q = 0; q < kPagePlanes; ++q)
        if (lane == q) {
            in = src.base[q];
            out = dst.base[q];
            stride = (int64_t)src.units[q] * 16;
            o0 = src.off[q];
            o1 = src.off[q + 1];
        }
    bool ok = true;
    int64_t i = blockIdx.x;  // the next piece, its page's move m
    int2 m = i < work ? at(i / chunks) : make_int2(-1, -1);
    int to[kRing], ch[kRing];  // of the pieces in the slots
    int loaded = 0, stored = 0;
    // kRing steps to the round, so that to and ch stay in registers
    for (bool more = true; more && ok;) {
#pragma unroll
        for (int s = 0; s < kRing; ++s) {
            while (i < work && m.y < 0) {  // pages that go nowhere
                i += ctas;
                if (i < work) m = at(i / chunks);
            }
            const bool load = ok && i < work;
            if (load) {
                const int64_t from = m.x;
                const int c = (int)(i % chunks), u0 = c * size, u1 = min(total, u0 + size);
                to[s] = m.y;
                ch[s] = c;
                i += ctas;
                if (i < work) m = at(i / chunks);  // on its way while the copies go out
                bulk_wait<1, true>();  // this lane's store that last used the slot has read it
                const uint32_t bar = bar0 + 8 * s, slot = ring + (uint32_t)(s * kCopyUnits * 16);
                if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(u1 - u0) * 16u);
                __syncwarp();
                const int a = max(u0, o0), b = min(u1, o1);
                if (a < b) bulk_g2s(slot + (uint32_t)(a - u0) * 16u, in + from * stride + (int64_t)(a - o0) * 16, (uint32_t)(b - a) * 16u, bar);
                ++loaded;
            }
            // store the oldest piece once the loads are kLag ahead of it, or done
            if (ok && stored < loaded && (loaded - stored > kLag || !load)) {
                const int n = stored % kRing;
                ok = __all_sync(TQ_FULL_MASK, mbar_wait_bounded(bar0 + 8 * n, (uint32_t)((stored / kRing) & 1), kWaitLimitNs,
                                                                 err, kErrPageWait));
                if (ok) {
                    int64_t t = 0;
                    int c = 0;
#pragma unroll
                    for (int z = 0; z < kRing; ++z)
                        if (z == n) {
                            t = to[z];
                            c = ch[z];
                        }
                    const int u0 = c * size, u1 = min(total, u0 + size);
                    const int a = max(u0, o0), b = min(u1, o1);
                    if (a < b)
                        bulk_s2g(out + t * stride + (int64_t)(a - o0) * 16, ring + (uint32_t)(n * kCopyUnits + a - u0) * 16u, (uint32_t)(b - a) * 16u);
                    bulk_commit();  // a group per piece and lane, empty or not
                    ++stored;
                }
            }
            if (!load && stored == loaded) more = false;
        }
    }
    // nothing is in flight when the CTA's shared memory goes: the loads still
    // out after a wait that ran out, then the stores
    for (int n = stored; n < loaded; ++n)
        mbar_wait_bounded(bar0 + 8 * (n % kRing), (uint32_t)((n / kRing) & 1), kWaitLimitNs, err, kErrPageWait);
    bulk_wait<0, false>();
}

__device__ __forceinline__ int64_t row_tokens(int n, const TableParams& t, int page) {
    return min((int64_t)max(n, 0), (int64_t)t.max_pages * page);
}

// ------------------------------------------------------------- many rows ---

// blocks[b] = the sum of f over block b of the rows: one CTA each
template <typename P>
__global__ void __launch_bounds__(kPageThreads) row_blocks_kernel(const __grid_constant__ P p) {
    static_assert(kRowBlock == kPageThreads, "a thread per row");
    wait_prior_grid();
    const int row = blockIdx.x * kRowBlock + (int)threadIdx.x;
    const int sum = block_sum(row < p.rows() ? p.asks(row) : 0);
    if (threadIdx.x == 0) p.blocks[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kPageThreads) fork_clear_kernel(const __grid_constant__ ForkParams p) {
    begin_call();
    const int r = blockIdx.x * kPageThreads + (int)threadIdx.x;
    if (r >= p.src.rows) return;
    p.first[r] = 0x7fffffff;
    p.children[r] = 0;
}

__global__ void __launch_bounds__(kPageThreads) fork_parents_kernel(const __grid_constant__ ForkParams p) {
    wait_prior_grid();
    const int i = blockIdx.x * kPageThreads + (int)threadIdx.x;
    if (i >= p.dst.rows) return;
    const int r = p.parent[i];
    if ((unsigned)r >= (unsigned)p.src.rows) return;
    atomicMin(p.first + r, i);
    atomicAdd(p.children + r, 1);
}

// ---------------------------------------------------------------- reserve ---

// Besides empty entries, a row asks for a page where its tokens go on in the
// middle of one that another entry holds too: written there, they would
// overwrite the other row's.

// The tokens [len, end) that a row adds and the pages [j0, j1) that they lie in:
// `part` tokens of page j0 are the row's already, `past` pages lie past the table.
// (Both numbers stay below 2^32: 32-bit divisions.)
struct RowRange {
    uint32_t len, end;
    int j0, j1, past, part;
};

__device__ __forceinline__ RowRange row_range(const ReserveParams& p, int row) {
    const uint32_t page = (uint32_t)p.pool.page, most = (uint32_t)p.t.max_pages;
    RowRange r;
    r.len = (uint32_t)max(p.lengths[row], 0);
    r.end = r.len + (uint32_t)max(p.add ? p.add[row] : p.add_all, 0);
    const uint32_t a = r.len / page, b = r.end > r.len ? (r.end - 1u) / page + 1u : a;
    r.j0 = (int)min(a, most);
    r.j1 = (int)min(b, most);
    r.past = (int)(b - max(a, min(b, most)));
    r.part = (int)(r.len - a * page);
    return r;
}

// granted: the row's tokens of [len, end) before page j1, the last, or `gap`, the
// first page that the row does not hold after the call (j1: there is none). In
// the page of its own last tokens that is as many below 0.
__device__ __forceinline__ int row_granted(const ReserveParams& p, const RowRange& r, int gap) {
    const int64_t page = p.pool.page;
    if (gap < r.j1) return (int)(gap * page - r.len);
    return (int)max((int64_t)0, min((int64_t)r.end, r.j1 * page) - r.len);
}

// CTAs [0, segs): the index; the others: one row each, its requests counted
__global__ void __launch_bounds__(kPageThreads) reserve_count_kernel(const __grid_constant__ ReserveParams p) {
    begin_call();
    if ((int)blockIdx.x < p.ix.segs) {
        index_segment(p.pool, p.ix, blockIdx.x);
        if (blockIdx.x == 0 && threadIdx.x == 0 && p.shortage) *p.shortage = 0;
        return;
    }
    // one warp per row
    const int row = (blockIdx.x - p.ix.segs) * (kPageThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= p.t.rows) return;
    const RowRange rr = row_range(p, row);
    int n = 0;
    bool own = false;  // lane 0: the half-filled last page is another entry's too, the row wants one of its own
    for (int j = rr.j0 + lane; j < rr.j1; j += 32) {
        const int e = p.t.e[row * p.t.stride + j];
        bool ask = !page_ok(e, p.pool.n_pages);
        if (j == rr.j0 && rr.part && !ask) ask = own = p.pool.refs[e] > 1;
        n += ask ? 1 : 0;
    }
    n = __reduce_add_sync(TQ_FULL_MASK, n);
    if (lane == 0) p.need[row] = 2 * n + (own ? 1 : 0);
}

// The first `tokens` tokens of page `pg` become zero vectors: their norms are 0
// (the planes of 2 bytes a slot), which nothing else of a slot outlives.
__device__ __forceinline__ void clear_tokens(const PoolParams& pool, int64_t pg, int tokens) {
    const int slots = pool.slots;
#pragma unroll
    for (int q = 0; q < kPagePlanes; ++q) {
        if (pool.units[q] != slots / 8) continue;
        uint16_t* x = reinterpret_cast<uint16_t*>(pool.base[q]) + pg * slots;
        for (int i = threadIdx.x; i < slots; i += kPageThreads)
            if (i % pool.page < tokens) x[i] = 0;
    }
}

// One CTA per row. A half-filled last page that another entry holds too is
// copied to the page the row takes for it (all of the row's holders decide by
// the counts as they stood, so where all of them take one the old page is free
// after the call); one that the row does not hold is cleared up to the row's
// length, since whatever the page held before would be seen there.
__global__ void __launch_bounds__(kPageThreads) reserve_take_kernel(const __grid_constant__ ReserveParams p) {
    extern __shared__ int s_pre[];
    __shared__ int s_from, s_to, s_gap;
    wait_prior_grid();
    const int row = blockIdx.x;
    const int need = p.need[row], want = need >> 1;
    const bool own = need & 1;
    const RowRange rr = row_range(p, row);
    if (threadIdx.x == 0) {
        if (rr.past > 0 && p.shortage) atomicAdd(p.shortage, rr.past);
        s_from = s_to = -1;
        s_gap = rr.j1;  // the first page the row does not hold after the call
        if (want == 0 && p.granted) p.granted[row] = row_granted(p, rr, rr.j1);
    }
    if (want == 0) return;
    load_prefix(p.ix, s_pre);
    int rank = rows_before(row, p.blocks, [&](int r) { return p.asks(r); });  // this row's first request
    const int free_pages = s_pre[p.ix.segs];
    for (int j = rr.j0; j < rr.j1; j += kPageThreads) {
        const int jj = j + (int)threadIdx.x;
        int32_t* e = p.t.e + row * p.t.stride + jj;
        const int old = jj < rr.j1 ? *e : -1;
        const bool copy = own && jj == rr.j0;
        const bool ask = jj < rr.j1 && (copy || !page_ok(old, p.pool.n_pages));
        int total;
        const int r = rank + block_prefix(ask ? 1 : 0, &total);
        if (ask) {
            int got = -1;
            if (r < free_pages) {
                got = find_free(p.ix, s_pre, r);
                p.pool.refs[got] = 1;
            } else {
                atomicMin(&s_gap, jj);
                if (p.shortage) atomicAdd(p.shortage, 1);
            }
            *e = got;
            if (jj == rr.j0 && rr.part) {
                if (copy) s_from = old;
                s_to = got;
            }
        }
        rank += total;
    }
    __syncthreads();
    if (threadIdx.x == 0 && p.granted) p.granted[row] = row_granted(p, rr, s_gap);
    const int from = s_from, to = s_to;
    if (to >= 0) {
        if (from < 0) clear_tokens(p.pool, to, rr.part);
        else
            for (int c = 0; c * kCopyUnits < p.pool.off[kPagePlanes]; ++c) copy_chunk(p.pool, p.pool, from, to, c);
    }
    if (from >= 0 && threadIdx.x == 0) atomicSub(p.pool.refs + from, 1);
}

// ------------------------------------------------------------------- fork ---

// Row i of dst from row r = parent[i] of src, n tokens: its full pages are
// shared; a half-filled last page and what was reserved behind it go to the
// first child where the row is given up, and every other child gets a copy of
// the half-filled page (taken by the second launch) and nothing behind it.
// CTAs [0, segs): the index; the others: one dst row each.
__global__ void __launch_bounds__(kPageThreads) fork_rows_kernel(const __grid_constant__ ForkParams p) {
    begin_call();
    if ((int)blockIdx.x < p.ix.segs) {
        index_segment(p.pool, p.ix, blockIdx.x);
        if (blockIdx.x == 0 && threadIdx.x == 0 && p.shortage) *p.shortage = 0;
        return;
    }
    const int i = blockIdx.x - p.ix.segs, r = p.parent[i];
    int32_t* out = p.dst.e + i * p.dst.stride;
    if ((unsigned)r >= (unsigned)p.src.rows) {  // no parent: an empty row
        for (int j = threadIdx.x; j < p.dst.max_pages; j += kPageThreads) out[j] = -1;
        if (threadIdx.x == 0) {
            p.tail[i] = -1;
            if (p.dst_lengths) p.dst_lengths[i] = 0;
        }
        return;
    }
    int earlier = 0;  // children of the same parent before this one
    if (p.first) earlier = p.first[r] != i;
    else
        for (int k = threadIdx.x; k < i; k += kPageThreads) earlier |= p.parent[k] == r;
    const bool heir = !__syncthreads_or(earlier) && !p.keep_src;
    const int64_t n = row_tokens(p.src_lengths[r], p.src, p.pool.page);
    const int full = (int)(n / p.pool.page);
    const bool part = n % p.pool.page != 0;
    const int32_t* in = p.src.e + r * p.src.stride;
    for (int j = threadIdx.x; j < p.dst.max_pages; j += kPageThreads) {
        int e = j < p.src.max_pages && (j < full || heir) ? in[j] : -1;
        out[j] = page_ok(e, p.pool.n_pages) ? e : -1;
    }
    if (threadIdx.x == 0) {
        const int e = part && !heir ? in[full] : -1;
        p.tail[i] = page_ok(e, p.pool.n_pages) ? e : -1;
        if (p.dst_lengths) p.dst_lengths[i] = (int)n;
    }
}

// CTAs [0, src.rows): the counts of one src row's pages; then `chunks` CTAs
// per dst row: its own copy of the half-filled page.
__global__ void __launch_bounds__(kPageThreads) fork_copy_kernel(const __grid_constant__ ForkParams p) {
    extern __shared__ int s_pre[];
    wait_prior_grid();
    if ((int)blockIdx.x < p.src.rows) {
        const int r = blockIdx.x;
        int children;
        if (p.children) {
            children = p.children[r];
        } else {
            int mine = 0;
            for (int k = threadIdx.x; k < p.dst.rows; k += kPageThreads) mine += p.parent[k] == r;
            children = block_sum(mine);
        }
        const int64_t n = row_tokens(p.src_lengths[r], p.src, p.pool.page);
        const int full = (int)(n / p.pool.page);
        // a row given up loses its own hold, which its first child takes over
        const int on_full = children - (p.keep_src ? 0 : 1);
        const int behind = !p.keep_src && children == 0 ? -1 : 0;
        int32_t* e = p.src.e + r * p.src.stride;
        for (int j = threadIdx.x; j < p.src.max_pages; j += kPageThreads) {
            const int d = j < full ? on_full : behind;
            if (d != 0 && page_ok(e[j], p.pool.n_pages)) atomicAdd(p.pool.refs + e[j], d);
            if (!p.keep_src) e[j] = -1;
        }
        return;
    }
    const int i = (blockIdx.x - p.src.rows) / p.chunks, c = (blockIdx.x - p.src.rows) % p.chunks;
    const int from = p.tail[i];
    if (from < 0) return;
    load_prefix(p.ix, s_pre);
    const int rank = rows_before(i, p.blocks, [&](int k) { return p.asks(k); });
    if (rank >= s_pre[p.ix.segs]) {
        if (c == 0 && threadIdx.x == 0 && p.shortage) atomicAdd(p.shortage, 1);
        return;
    }
    const int to = find_free(p.ix, s_pre, rank);  // every thread: the same loads
    copy_chunk(p.pool, p.pool, from, to, c);
    if (c == 0 && threadIdx.x == 0) {
        const int64_t n = row_tokens(p.src_lengths[p.parent[i]], p.src, p.pool.page);
        p.dst.e[i * p.dst.stride + n / p.pool.page] = to;
        p.pool.refs[to] = 1;
    }
}

// ------------------------------------------------------------------- trim ---

// one thread per table entry
__global__ void __launch_bounds__(kPageThreads) trim_kernel(const __grid_constant__ TrimParams p) {
    begin_call();
    const int per_row = (p.t.max_pages + kPageThreads - 1) / kPageThreads;
    const int row = blockIdx.x / per_row, j = (blockIdx.x - row * per_row) * kPageThreads + threadIdx.x;
    if (j >= p.t.max_pages) return;
    int32_t* e = p.t.e + row * p.t.stride + j;
    const int held = *e;
    const int64_t n = max(p.lengths[row], 0), page = p.pool.page;
    const int64_t low = p.window > 0 ? n - p.window : 0;
    const bool gone = j * page >= n || (j * page >= p.sinks && (j + 1) * page <= low);
    if (gone && page_ok(held, p.pool.n_pages)) {
        *e = -1;
        atomicSub(p.pool.refs + held, 1);
    }
}

// ------------------------------------------------------------------- copy ---

__global__ void __launch_bounds__(32) copy_kernel(const __grid_constant__ CopyParams p) {
    stream_pages(p.src, p.dst,
                 [&](int64_t i) {
                     const int from = p.from[i], to = p.to[i];
                     return page_ok(from, p.src.n_pages) && page_ok(to, p.dst.n_pages) ? make_int2(from, to) : make_int2(-1, -1);
                 },
                 (int64_t)p.n * p.chunks, p.chunks, p.ctas, p.err);
}

// ---------------------------------------------------------------- compact ---

__global__ void __launch_bounds__(kPageThreads) compact_index_kernel(const __grid_constant__ CompactParams p) {
    begin_call();
    index_segment(p.src, p.ix, blockIdx.x);
}

// One thread per page: where it goes. With L live pages, page p < L stays and
// the i-th live page from L on takes the i-th lowest free page (those all lie
// below L). The list of moves holds the pages that move (in place) or all live
// ones (into another pool), in page order.
__global__ void __launch_bounds__(kPageThreads) compact_map_kernel(const __grid_constant__ CompactParams p) {
    extern __shared__ int s_pre[];
    let_next_grid();
    wait_prior_grid();
    load_prefix(p.ix, s_pre);
    const int n = p.src.n_pages;
    const int live = n - s_pre[p.ix.segs];
    const int holes = free_below(p.ix, s_pre, live);  // = the live pages from `live` on
    const int64_t q = (int64_t)blockIdx.x * kPageThreads + threadIdx.x;
    if (q < n) {
        const int pg = (int)q;
        const int fb = free_below(p.ix, s_pre, pg);
        const bool is_free = (p.ix.bits[pg >> 5] >> (pg & 31)) & 1u;
        int to = -1;
        if (!is_free) {
            const int i = (pg - fb) - (live - holes);  // its rank among the live pages from `live` on
            to = pg < live ? pg : find_free(p.ix, s_pre, i);
            if (to >= p.dst.n_pages) to = -1;  // the other pool is too small
            if (!p.in_place) p.move[pg - fb] = make_int2(pg, to);
            else if (pg >= live) p.move[i] = make_int2(pg, to);
        }
        p.map[pg] = to;
    }
    // pages of the other pool that hold nothing
    if (!p.in_place)
        for (int64_t q = live + (int64_t)blockIdx.x * kPageThreads + threadIdx.x; q < p.dst.n_pages;
             q += (int64_t)gridDim.x * kPageThreads)
            p.dst.refs[q] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *p.n_move = p.in_place ? holes : live;
        if (p.live) *p.live = live;
    }
}

// Warp 0 of each CTA streams the pages, the others move the counts and rewrite
// the tables.
__global__ void __launch_bounds__(kPageThreads) compact_move_kernel(const __grid_constant__ CompactParams p) {
    wait_prior_grid();
    const int moves = *p.n_move;
    if (threadIdx.x < 32) {
        stream_pages(p.src, p.dst, [&](int64_t i) { return p.move[i]; }, (int64_t)moves * p.chunks, p.chunks, p.ctas, p.err);
        return;
    }
    const int64_t first = (int64_t)blockIdx.x * (kPageThreads - 32) + threadIdx.x - 32;
    const int64_t step = (int64_t)gridDim.x * (kPageThreads - 32);
    for (int64_t i = first; i < moves; i += step) {
        const int2 m = p.move[i];
        if (m.y < 0) continue;
        p.dst.refs[m.y] = p.src.refs[m.x];
        if (p.in_place) p.src.refs[m.x] = 0;
    }
#pragma unroll
    for (int t = 0; t < kMaxPageTables; ++t) {
        if (t >= p.n_tables) break;
        const int mp = p.from[t].max_pages;
        const int64_t entries = (int64_t)p.from[t].rows * mp;
        for (int64_t i = first; i < entries; i += step) {
            const int64_t row = i / mp, j = i - row * mp;
            const int e = p.from[t].e[row * p.from[t].stride + j];
            p.to[t].e[row * p.to[t].stride + j] = page_ok(e, p.src.n_pages) ? p.map[e] : -1;
        }
    }
}

// a launch that may start while the one before it on the stream finishes (its
// CTAs wait for that one before they read anything)
template <typename P>
cudaError_t launch_after(void (*kernel)(P), unsigned ctas, size_t smem, const P& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPageThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

unsigned ctas_of(int rows) { return (unsigned)((rows + kPageThreads - 1) / kPageThreads); }

size_t prefix_smem(const PageIndex& ix) { return (size_t)(ix.segs + 1) * sizeof(int); }

}  // namespace

int page_copy_chunks(int units) { return (units + kCopyUnits - 1) / kCopyUnits; }

cudaError_t launch_pages_reserve(const ReserveParams& p, cudaStream_t s) {
    if (p.t.rows <= 0) return cudaSuccess;
    const unsigned row_ctas = (unsigned)((p.t.rows + kPageThreads / 32 - 1) / (kPageThreads / 32));
    cudaError_t e = launch_after(reserve_count_kernel, (unsigned)p.ix.segs + row_ctas, 0, p, s);
    if (e != cudaSuccess) return e;
    if (p.blocks && (e = launch_after(row_blocks_kernel<ReserveParams>, ctas_of(p.t.rows), 0, p, s)) != cudaSuccess) return e;
    return launch_after(reserve_take_kernel, (unsigned)p.t.rows, prefix_smem(p.ix), p, s);
}

cudaError_t launch_pages_fork(const ForkParams& p, cudaStream_t s) {
    cudaError_t e;
    if (p.first && p.src.rows > 0) {
        if ((e = launch_after(fork_clear_kernel, ctas_of(p.src.rows), 0, p, s)) != cudaSuccess) return e;
        if ((e = launch_after(fork_parents_kernel, ctas_of(p.dst.rows), 0, p, s)) != cudaSuccess) return e;
    }
    if ((e = launch_after(fork_rows_kernel, (unsigned)(p.ix.segs + p.dst.rows), 0, p, s)) != cudaSuccess) return e;
    if (p.blocks && (e = launch_after(row_blocks_kernel<ForkParams>, ctas_of(p.dst.rows), 0, p, s)) != cudaSuccess) return e;
    if (p.src.rows <= 0 && p.dst.rows <= 0) return cudaSuccess;
    return launch_after(fork_copy_kernel, (unsigned)(p.src.rows + p.dst.rows * p.chunks), prefix_smem(p.ix), p, s);
}

cudaError_t launch_pages_trim(const TrimParams& p, cudaStream_t s) {
    if (p.t.rows <= 0) return cudaSuccess;
    const int64_t ctas = (int64_t)p.t.rows * ((p.t.max_pages + kPageThreads - 1) / kPageThreads);
    if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_after(trim_kernel, (unsigned)ctas, 0, p, s);
}

cudaError_t launch_pages_copy(const CopyParams& p, cudaStream_t s) {
    if (p.n <= 0) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes);
    if (e != cudaSuccess) return e;
    copy_kernel<<<(unsigned)p.ctas, 32, kRingBytes, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_pages_compact(const CompactParams& p, cudaStream_t s) {
    cudaError_t e = launch_after(compact_index_kernel, (unsigned)p.ix.segs, 0, p, s);
    if (e != cudaSuccess) return e;
    if ((e = launch_after(compact_map_kernel, (unsigned)((p.src.n_pages + kPageThreads - 1) / kPageThreads), prefix_smem(p.ix), p, s)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(compact_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes)) != cudaSuccess)
        return e;
    return launch_after(compact_move_kernel, (unsigned)p.ctas, kRingBytes, p, s);
}

}  // namespace tqk
