// Windowed / paged chunked-prefill attention on the 5th-generation tensor
// cores, for keys at 1 or 2 code bits (PROD 2 or 3 bits, or the 3 / 2
// fractional rate).
//
// The mathematics of prefill_umma.cuh (A2A TurboQuant explainer, end of
// "Stage 2"; Qiita TurboQuant article, "One more stage ..."): S = Q Bs^T per
// 128-token tile, an online softmax over its rows, O += P V, with 128 query
// rows per unit and the units' tiles dealt out evenly (stream-K). A unit's
// tiles are the 128-token tiles that any of its rows sees (view.cuh); rows are
// masked to their own window, the sinks and the pages that hold something.
//
// What bounds it: the softmax warps. Per tile (5.9 K cycles in the kernel this
// one started from) they were busy for 5.2 K, the key warps for 3.8 K, the
// value warps for 2.8 K and the tensor pipe for 1.9 K, and the code was 107 KB,
// several times the instruction cache. Hence, against prefill_umma.cuh:
//  * a row's reference R (what its exponents are taken against) is not its
//    running maximum but moves only when a weight could leave fp16's range, so
//    O is rescaled in a tile or two of a segment, not in most of them;
//  * the two threads of a row meet once per tile, on a hardware barrier;
//  * for a bf16 output P has one fp16 limb and the sign part's query one, q'
//    keeps two: a weight is then off by at most 2^-11 of itself and a logit by
//    about 1e-4 of ||q|| n / sqrt(d) (the sign part's rounding); over the tokens
//    of a window that averages to well under the 2^-9 of the output's own
//    rounding. All of the query operand lives in TMEM then, and the place of its
//    lo limbs in shared memory takes a second Bs buffer, so that the next tile's
//    keys are written while this one's scores are formed. For an fp32 output (FL)
//    P and both parts of the query have two limbs, the query's lo limbs in shared
//    memory and one Bs buffer, as in prefill_umma.cuh: the scan of 512 tokens
//    behind 4096 then takes 110 us where the bf16 form takes 90, the call 127
//    against 107 us (L2 flushed), two chunks of 2048 behind 8192 1.42 against 1.27 ms;
//  * cold code is rolled and a wait is a handful of instructions;
//  * the shared-memory pipe was 90 % busy with table lookups, operand stores and
//    the tensor cores' reads (4.5 K of 5.0 K cycles a tile): 2-bit key codes
//    become fp16 pairs by byte permutes instead of lookups, and the value tables
//    hold a copy of each entry per bank.
// Measured (GB300, K3 / V3, 32 query / 8 KV heads, bf16 output): a 512-token chunk
// over 32768 tokens in full 491 us for the scan (prefill_umma.cuh 615), over 8192
// 145 us, behind a window of 4096 tokens 90 us (the call 99.7 us); two 2048-token
// chunks behind 8192 tokens with 4-bit values 1.24 ms, with 3-bit ones 1.06 ms.
// What bounds it now: the chain of a tile's values, about 3 K cycles for two warps
// to write V after O has read the one before (the instructions of its lookups),
// then 1.0 K for O. (V in four more warps' spare time, two groups at a time, a
// group ahead in registers, or in halves of 64 tokens was each slower: more
// instructions, more code in flight.)
//
// fp16 weights: P = 2^(l - R) nV with l in log2 units. nV goes into the
// exponent: the scores' factor is followed by log2 nV, P = 2^(l + log2 nV - R)
// comes out of one exponential, and Z = sum 2^(l - R) adds P / nV. R is raised
// to max(l + log2 nV) - 9 over the tokens that the row sees as soon as that
// maximum exceeds R by 15: P stays below 2^15, and a row's largest weights
// start near 2^9, 23 binades above fp16's last normal, whatever the norms are
// and whatever the tokens that it does not see hold. M = R and Z go to the
// merge, which only needs them to belong together. (Taking R from the largest
// nV of the tile instead let a large norm at an unseen token push the weights
// of small ones into fp16's subnormals. The third factor that the softmax reads
// per token, 1 / nV, costs 2.6 % where 4-bit values keep shared memory busiest:
// two 2048-token chunks 1.23 -> 1.26 ms a call.) A norm of 0 counts as 2^-64; one that
// is not finite, or negative, makes the rows that see it NaN.
//
// Pages: warp 14 looks up the pages of a tile's 16-token pieces, lane k for
// piece k, loaded one tile ahead, and fetches each run of pieces that follow one
// another with one copy per plane. It does nothing else: this takes it 2.2 K
// cycles a tile, and took 1.2 K of the thread that feeds the tensor cores (which
// has no time for it), while two warps write V in about 3 K.
//
// Warp roles: 0-7 softmax (two threads per row), 8-11 Bs (thread = token), 12
// and 13 V, 14 copies, 15 MMA issue (one thread).
#pragma once

#include "prefill_umma.cuh"

namespace tqk {

constexpr float kNoNorm = 5.421010862427522e-20f;  // 2^-64, in place of a value norm of 0
constexpr uint32_t kVwColP = 384;    // TMEM: P (64 columns); Q, S and O as in prefill_umma.cuh
constexpr uint32_t kVwColQlo = 448;  // lo limb of q' (64 columns)
constexpr uint32_t kVwColPlo = 448;  // FL: lo limb of P in its place

// The bounded wait of the other kernels in a handful of instructions a site: the
// clock is read at every poll, which only a wait that did not succeed at once
// takes part in.
__device__ __forceinline__ bool vw_wait(uint32_t bar, uint32_t parity, uint32_t* err) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
#pragma unroll 1
    do {
        __nanosleep(64);
        if (mbar_try_wait(bar, parity)) return true;
    } while (global_ns() - t0 < kWaitLimitNs);
    if (err) atomicOr(err, kErrScanWait);
    return false;
}

// The n lowest bits (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// A unit's share of the CTA's run of tiles: query block qb of KV head kv of
// batch row b, visible tiles v0 .. v0 + ntiles - 1 of the unit; lim the end of
// the tokens its last row sees, nst / wt0 / sink_end its ViewTiles and the end of
// the tokens that the last tile of the sinks needs; tg0 the CTA's tiles before
// it; the unit's rows' partials go to slot, of nslot.
struct VwSeg {
    int qb, b, kv;
    int v0, ntiles, tg0, slot, nslot;
    int lim, nst, wt0, sink_end;
};

__device__ __forceinline__ int vw_token(const VwSeg& sg, int T) {
    const int v = sg.v0 + T;
    return (v < sg.nst ? v : v - sg.nst + sg.wt0) * kPuTok;
}

// sync of the two warps of a row's pair with an or over their threads
__device__ __forceinline__ bool pair_sync_or(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, %2, 64, q;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(r)
        : "r"(v ? 1u : 0u), "r"(id)
        : "memory");
    return r != 0;
}

// Copies of a value pair table of n entries (8 KB in all; two tables share it).
constexpr int vw_copies(int n, bool two) {
    const int c = (two ? 1024 : 2048) / n;
    return c > 32 ? 32 : c;
}

// A stage and its per-token factors: of the scores, log2 nV and 1 / nV.
template <typename ST>
constexpr int vw_stage_bytes() {
    return ST::OFF_FK + 3 * kPuTok * 4;
}

constexpr int vw_log2(int n) { return n <= 1 ? 0 : 1 + vw_log2(n / 2); }

// FL: the caller's output is fp32 (see the top).
template <int KB, int VB, int KB2, int VB2, bool FL>
__global__ void __launch_bounds__(kPuThreads, 1) prefill_view_kernel(const __grid_constant__ PrefillParams p) {
    using ST = PuStage<KB, VB, KB2, VB2>;
    constexpr int SB = vw_stage_bytes<ST>();
    constexpr bool K2 = KB2 != KB, V2 = VB2 != VB;
    constexpr int KL = 1 << (2 * KB), VL = 1 << (2 * VB);
    constexpr int KL2 = K2 ? 1 << (2 * KB2) : 1, VL2 = V2 ? 1 << (2 * VB2) : 1;
    constexpr int D = 128;

    extern __shared__ __align__(1024) unsigned char vw_smem[];
    constexpr int NB = FL ? 1 : 2;                 // buffers of Bs
    unsigned char* sBs = vw_smem;
    unsigned char* sQlo = sBs + kPuBsBytes;        // FL: the lo limbs of the query operand
    unsigned char* sV = sBs + 2 * kPuBsBytes;
    static_assert(kPuQloBytes == kPuBsBytes, "the lo limbs take the second buffer's place");
    unsigned char* ring = sV + kPuVBytes;

    __shared__ uint32_t klut[KL];
    __shared__ uint32_t klut2[KL2];
    // 2-bit keys at one width: four codes at a time by byte permutes (below)
    constexpr bool KQ = KB == 2 && !K2;
    // the value pair tables, VC (VC2) copies of each entry side by side, lane l
    // reading copy l % VC: with 32 copies every lane has a bank of its own
    constexpr int VC = vw_copies(VL, V2), VC2 = vw_copies(VL2, V2);
    __shared__ uint32_t vlut[VL * VC];
    __shared__ uint32_t vlut2[V2 ? VL2 * VC2 : 1];
    __shared__ float s_max[2][2][kPuRows];         // a row's two column halves, alternating by tile
    __shared__ int2 s_rows[kPuRows];               // each row's window [x, y) in the current segment
    __shared__ uint32_t s_held[kPuStages];         // bit per 16 tokens of a stage whose page holds them
    __shared__ __align__(8) uint64_t s_bar[3 * kPuStages + 10];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ VwSeg s_seg[kPuMaxSegView];
    __shared__ int s_nseg, s_ntot;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = p.group;

    const uint32_t bar0 = (uint32_t)__cvta_generic_to_shared(&s_bar[0]);
    auto bar_at = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    auto ring_full = [&](int s) { return bar_at(s); };
    auto ring_empty = [&](int s) { return bar_at(kPuStages + s); };
    auto fac_full = [&](int s) { return bar_at(2 * kPuStages + s); };
    auto bs_full = [&](int b) { return bar_at(3 * kPuStages + b); };      // Bs(T) written to buffer T % NB (4 warps)
    auto bs_free = [&](int b) { return bar_at(3 * kPuStages + 2 + b); };  // and read (commit)
    const uint32_t s_done = bar_at(3 * kPuStages + 4);    // S(T) complete (commit)
    const uint32_t v_full = bar_at(3 * kPuStages + 5);    // V(T) written (2 warps)
    const uint32_t o_done = bar_at(3 * kPuStages + 6);    // O += P(T) V(T) complete (commit)
    const uint32_t s_empty = bar_at(3 * kPuStages + 7);   // S(T) read by the softmax (8 warps)
    const uint32_t p_full = bar_at(3 * kPuStages + 8);    // P(T) written, O rescaled (8 warps)
    const uint32_t q_full = bar_at(3 * kPuStages + 9);    // A of S in TMEM (8 warps)

    fill_pairs<KB>(klut, p.klut);
    if constexpr (K2) fill_pairs<KB2>(klut2, p.klut2);
    // the value tables from their first entries too (fill_pairs of decode_mma.cuh)
    auto fill_copies = [&](uint32_t* dst, const uint32_t* src, int bits, int copies) {
        const int n = 1 << bits;
        const uint32_t first = src[lane & (n - 1)];
#pragma unroll 1
        for (int i = tid; i < n * n * copies; i += kPuThreads) {  // a multiple of 32 in all
            const int e = i / copies;
            dst[i] = prmt(__shfl_sync(TQ_FULL_MASK, first, e & (n - 1)), __shfl_sync(TQ_FULL_MASK, first, e >> bits), 0x5410u);
        }
    };
    fill_copies(vlut, p.vlut, VB, VC);
    if constexpr (V2) fill_copies(vlut2, p.vlut2, VB2, VC2);
    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < 3 * kPuStages + 10; ++i) {
            // arrivals: the ring's consumers are 4 Bs + 2 V + 8 softmax warps
            const int j = i - 3 * kPuStages;
            const int n = i < kPuStages ? 1 : i < 2 * kPuStages ? 14 : i < 3 * kPuStages ? 4
                          : j < 2 ? 4 : j == 5 ? 2 : (j == 7 || j == 8 || j == 9) ? 8 : 1;
            mbar_init(bar_at(i), (uint32_t)n);
        }
        s_abort = 0;
        mbar_init_fence();
        // this CTA's segments: tiles [g0, g1) of the (unit, tile) sequence
        const int64_t total = (int64_t)p.qbs * p.batch * p.hkv * p.unit_tiles;
        const int64_t g0 = (int64_t)blockIdx.x * p.tiles_per_cta;
        const int64_t g1 = min(g0 + p.tiles_per_cta, total);
        int n = 0, tg = 0;
        int64_t g = g0;
#pragma unroll 1
        for (; g < g1 && n < kPuMaxSegView; ++n) {
            const int64_t u = g / p.unit_tiles;
            const int a = (int)(g - u * p.unit_tiles);
            const int bend = (int)min((int64_t)p.unit_tiles, a + (g1 - g));
            VwSeg sg;
            sg.qb = (int)(u % p.qbs);
            const int bkv = (int)(u / p.qbs);
            sg.b = bkv / p.hkv;
            sg.kv = bkv % p.hkv;
            // the unit's tiles: its first row's window to its last row's position
            const int start = p.q_start[sg.b], i0 = sg.qb * kPuRows / G;
            const int i1 = min(p.chunk - 1, (sg.qb * kPuRows + kPuRows - 1) / G);
            sg.lim = max(0, min(start + i1 + 1, p.lim_cap));
            const int low = view_low(p.view, start + i0 + 1);
            ViewTiles<kPuTok> vt;
            vt.init(p.view.sinks, low, sg.lim);
            sg.v0 = a;
            sg.ntiles = max(0, min(bend, vt.nv) - a);
            sg.nst = vt.nst;
            sg.wt0 = vt.wt0;
            sg.sink_end = low >= vt.nst * kPuTok ? vt.sinks : sg.lim;
            sg.tg0 = tg;
            const int64_t fc = (u * p.unit_tiles) / p.tiles_per_cta;
            sg.slot = (int)(blockIdx.x - fc);
            sg.nslot = (int)(((u + 1) * p.unit_tiles - 1) / p.tiles_per_cta - fc + 1);
            s_seg[n] = sg;
            tg += sg.ntiles;
            g += bend - a;
        }
        if (g < g1) {  // more units than the plan allows (the host bounds it): report, do nothing
            if (p.err) atomicOr(p.err, kErrScanWait);
            n = 0;
            tg = 0;
        }
        s_nseg = n;
        s_ntot = tg;
    }
    if (warp == 15) {
        tmem_alloc((uint32_t)__cvta_generic_to_shared(&s_tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = s_tmem;
    volatile int* abort_flag = &s_abort;

    const int nseg = s_nseg;
    const int ntot = s_ntot;
    const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
    const uint32_t v_s = (uint32_t)__cvta_generic_to_shared(sV);
    const uint32_t bs_s = (uint32_t)__cvta_generic_to_shared(sBs);
    const uint32_t qlo_s = (uint32_t)__cvta_generic_to_shared(sQlo);
    auto bs_buf = [&](int T) { return bs_s + (uint32_t)(T % NB) * (uint32_t)kPuBsBytes; };

    if (warp == 15) {
        // ======================= MMA issue (one thread) =======================
        if (lane == 0 && ntot > 0) {
            bool ok = true;
            const uint32_t idesc = umma_idesc_f16(kPuRows, kPuTok);
            int qn = 0, last_s = -1, last_o = -1;  // segments whose query operands were loaded; tiles issued
            for (int si = 0; ok && si < nseg; ++si) {
                const int nt = s_seg[si].ntiles, tg0 = s_seg[si].tg0;
                if (nt == 0) continue;
                // the softmax warps loaded this segment's query operands
                if (!(ok = vw_wait(q_full, (uint32_t)(qn & 1), p.err))) break;
                ++qn;
                // step T issues the scores of tile T, then O of tile T - 1: the
                // scores go in while the softmax works on the tile before
#pragma unroll 1
                for (int T = 0; T <= nt; ++T) {
                    const int Tg = tg0 + T;
                    if (*abort_flag) {
                        ok = false;
                        break;
                    }
                    if (T < nt) {
                        // S(T) = Q Bs(T)^T over K = 256: the key part (k-steps 0 .. 7)
                        // against both limbs of q', the sign part against kappa lam_k u
                        // (FL: both limbs, the lo ones from shared memory)
                        ok = vw_wait(bs_full(Tg % NB), (uint32_t)((Tg / NB) & 1), p.err) &&
                             (Tg == 0 || vw_wait(s_empty, (uint32_t)((Tg - 1) & 1), p.err));
                        if (!ok) break;
                        tc_fence_after_sync();
                        const uint32_t b0 = bs_buf(Tg);
#pragma unroll 1
                        for (int k = 0; k < 8; ++k) {
                            const uint64_t bk = umma_desc(b0 + 256u * k, 128, 4096), bz = umma_desc(b0 + 256u * (8 + k), 128, 4096);
                            umma_f16_ta(tmem + kPuColS, tmem + kPuColQ + 8u * k, bk, idesc, k > 0);
                            if constexpr (FL) umma_f16(tmem + kPuColS, umma_desc(qlo_s + 256u * k, 128, 4096), bk, idesc, true);
                            else umma_f16_ta(tmem + kPuColS, tmem + kVwColQlo + 8u * k, bk, idesc, true);
                            umma_f16_ta(tmem + kPuColS, tmem + kPuColQ + 64u + 8u * k, bz, idesc, true);
                            if constexpr (FL) umma_f16(tmem + kPuColS, umma_desc(qlo_s + 256u * (8 + k), 128, 4096), bz, idesc, true);
                        }
                        umma_commit(s_done);
                        umma_commit(bs_free(Tg % NB));
                        last_s = Tg;
                    }
                    if (T > 0) {
                        // O += P(T - 1) V(T - 1) over K = 128 tokens; the segment's
                        // first tile starts O afresh
                        ok = vw_wait(p_full, (uint32_t)((Tg - 1) & 1), p.err) && vw_wait(v_full, (uint32_t)((Tg - 1) & 1), p.err);
                        if (!ok) break;
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int k = 0; k < 8; ++k) {
                            const uint64_t bd = umma_desc(v_s + 256u * k, 128, 2048);
                            umma_f16_ta(tmem + kPuColO, tmem + kVwColP + 8u * k, bd, idesc, T > 1 || k > 0);
                            if constexpr (FL) umma_f16_ta(tmem + kPuColO, tmem + kVwColPlo + 8u * k, bd, idesc, true);
                        }
                        umma_commit(o_done);
                        last_o = Tg - 1;
                    }
                }
            }
            if (!ok) *abort_flag = 1;
            // everything issued completes (bounded) before TMEM and shared memory
            // are released: the last commits cover all MMAs before them
            if (last_s >= 0) {
                vw_wait(s_done, (uint32_t)(last_s & 1), p.err);
                vw_wait(bs_free(last_s % NB), (uint32_t)((last_s / NB) & 1), p.err);
            }
            if (last_o >= 0) vw_wait(o_done, (uint32_t)(last_o & 1), p.err);
        }
    } else if (warp == 14) {
        // ======================= bulk copies (the warp) =======================
        // the CTA's next tile is tile ct of segment cs; lane k < 8 holds its piece k
        // (tokens tok .. tok + 15, wanted when tok < end) and the page entry of it,
        // loaded one tile ahead
        int cs = -1, ct = 0, cnt = 0;
        int tok = 0, end = 0, row = 0, entry = -1, off = 0;  // row: b * hkv + kv (contiguous), kv (paged)
        auto look_ahead = [&]() {
#pragma unroll 1
            while (ct >= cnt) {
                if (cs + 1 >= nseg) return;
                cnt = s_seg[++cs].ntiles;
                ct = 0;
            }
            const VwSeg& sg = s_seg[cs];
            const int tb = vw_token(sg, ct);
            end = min(tb + kPuTok, sg.v0 + ct == sg.nst - 1 ? sg.sink_end : sg.lim);
            tok = tb + 16 * (lane & 7);
            row = sg.kv;
            ++ct;
            if (p.view.table != nullptr) {
                const int j = tok / p.view.page;
                off = tok - j * p.view.page;
                entry = j < p.view.max_pages ? __ldg(p.view.table + sg.b * p.view.table_stride + j) : -1;
            } else {
                row += sg.b * p.hkv;
            }
        };
        look_ahead();
        bool ok = true;
        // one bulk copy per plane and run of pieces, issued by the lane of the
        // run's first piece as soon as the softmax, Bs and V warps are done with
        // the tile that is in the stage
#pragma unroll 1
        for (int issued = 0; issued < ntot; ++issued) {
            const int s = issued % kPuStages;
            int64_t slot = -1;
            if (lane < 8 && tok < end) {
                if (p.view.table == nullptr) slot = row * p.capacity + tok;
                else if ((unsigned)entry < (unsigned)p.view.n_pages)
                    slot = ((int64_t)entry * p.hkv + row) * p.view.page + off;
            }
            const int64_t before = __shfl_up_sync(TQ_FULL_MASK, slot, 1);
            const bool first = slot >= 0 && (lane == 0 || before < 0 || slot != before + 16);
            const uint32_t held = __ballot_sync(TQ_FULL_MASK, slot >= 0), firsts = __ballot_sync(TQ_FULL_MASK, first);
            const uint32_t n = 16u * (uint32_t)__ffs((int)((firsts | ~held) >> (lane + 1)));  // tokens of the run
            const uint32_t bar = ring_full(s), st = ring_s + (uint32_t)(s * SB), at = 16u * (uint32_t)lane;
            look_ahead();
            const int T = issued - kPuStages;
            ok = T < 0 || (!*abort_flag && vw_wait(ring_empty(s), (uint32_t)((T / kPuStages) & 1), p.err));
            if (!__all_sync(TQ_FULL_MASK, ok)) {
                *abort_flag = 1;
                ok = false;
                // every copy issued lands (bounded) before the shared memory is released
#pragma unroll 1
                for (int t = max(0, T); t < issued; ++t)
                    vw_wait(ring_full(t % kPuStages), (uint32_t)((t / kPuStages) & 1), p.err);
                break;
            }
            // (no proxy fence: the stage's earlier readers released it through
            // ring_empty, and nothing wrote it since but copies)
            if (lane == 0) {
                s_held[s] = held;  // read by the Bs and softmax warps after their waits
                mbar_arrive_expect_tx(bar, 16u * (uint32_t)__popc(held) * (uint32_t)(ST::KS + 16 + 2 + 2 + ST::VS + 2));
            }
            __syncwarp();
            if (first) {
                bulk_g2s(st + ST::OFF_KC + at * ST::KS, p.kcodes + slot * ST::KS, n * ST::KS, bar);
                bulk_g2s(st + ST::OFF_SG + at * 16, p.ksigns + slot * 16, n * 16, bar);
                bulk_g2s(st + ST::OFF_KN + at * 2, p.knorm + slot, n * 2, bar);
                bulk_g2s(st + ST::OFF_KR + at * 2, p.krnorm + slot, n * 2, bar);
                bulk_g2s(st + ST::OFF_VC + at * ST::VS, p.vcodes + slot * ST::VS, n * ST::VS, bar);
                bulk_g2s(st + ST::OFF_VN + at * 2, p.vnorm + slot, n * 2, bar);
            }
            __syncwarp();
        }
        if (ok)
#pragma unroll 1
            for (int t = max(0, ntot - kPuStages); t < ntot; ++t)
                vw_wait(ring_full(t % kPuStages), (uint32_t)((t / kPuStages) & 1), p.err);
    } else if (warp >= 12) {
        // ======================= V: values through stmatrix =======================
        // warp vw writes token groups J (8 tokens each), the fragments those of
        // prefill_umma.cuh
        const int vw = warp - 12;
        const int q = lane & 3;
        constexpr int VN = ST::VS / 4;
        const uint32_t* vtab = vlut + lane % VC;
        const uint32_t* vtab2 = vlut2 + (V2 ? lane % VC2 : 0);
        const uint32_t copy4 = 4u * (lane % VC), copy4_2 = 4u * (lane % VC2);  // this lane's copy of an entry
        // this warp's token groups
        const int J0 = 8 * vw, J1 = J0 + 8;
#pragma unroll 1
        for (int T = 0; T < ntot; ++T) {
            const int s = T % kPuStages;
            bool ok = !*abort_flag && vw_wait(ring_full(s), (uint32_t)((T / kPuStages) & 1), p.err);
            // O += P(T - 1) V(T - 1) has read V(T - 1)
            if (ok && T > 0) ok = vw_wait(o_done, (uint32_t)((T - 1) & 1), p.err);
            if (!__all_sync(TQ_FULL_MASK, ok)) {
                *abort_flag = 1;
                break;
            }
            const unsigned char* st = ring + s * SB;
            uint32_t w[VN + 1];
            // the code words of this thread's token in group J
            auto load_row = [&](int J) {
                const unsigned char* vr = st + ST::OFF_VC + (8 * J + (lane >> 2)) * ST::VS;
                if constexpr (ST::VS % 16 == 0) {
#pragma unroll
                    for (int i = 0; i < VN / 4; ++i) {
                        const uint4 x = reinterpret_cast<const uint4*>(vr)[i];
                        w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < VN / 2; ++i) {
                        const uint2 x = reinterpret_cast<const uint2*>(vr)[i];
                        w[2 * i] = x.x; w[2 * i + 1] = x.y;
                    }
                }
                w[VN] = 0u;
            };
            load_row(J0);
#pragma unroll 1
            for (int J = J0; J < J1; ++J) {
                // Stale tokens index the tables like any other, so their values
                // are finite; their P is exactly 0. The loads are unconditional.
                uint32_t f[16];
#pragma unroll
                for (int bb = 0; bb < 16; ++bb) {
                    const bool first = !V2 || (bb & 1) == 0;
                    const int wd = first ? VB : VB2;
                    const int sc = 2 + vw_log2(first ? VC : VC2);  // an entry's copies are 2^sc bytes
                    // lane q's pair is the 2 wd bits from bit base + 2 wd q on; one shift
                    // takes them to bit sc where it can, and one three-way logical
                    // instruction masks them and adds the lane's copy (K3 / V3, 512
                    // tokens over 8192: 149.5 -> 143.4 us). 4-bit codes, whose lookups
                    // meet on banks, are better spread out by two shifts (1.20 ms
                    // against 1.25 ms at two chunks of 2048 behind 8192).
                    const int base = code_bit<VB, VB2>(8 * bb), k = base >> 5, b = base & 31;
                    uint32_t t;
                    if (wd == 4) {
                        t = b == 0 ? w[k] : __funnelshift_r(w[k], w[k + 1], b);
                        f[bb] = lds_at<uint32_t>(first ? vtab : vtab2, ((t >> (2 * wd * q)) & 0xFFu) << sc);
                        continue;
                    } else if (b + 8 * wd <= 32) {  // in one word for every q
                        t = __funnelshift_r(w[k], w[k], (uint32_t)(b - sc + 2 * wd * q));
                    } else if (b >= sc && b - sc + 6 * wd < 32) {
                        t = __funnelshift_r(w[k], w[k + 1], (uint32_t)(b - sc + 2 * wd * q));
                    } else {
                        const int c = 8;  // below 32 with 2 wd q, wd <= 3
                        t = __funnelshift_r(w[k], w[k + 1], (uint32_t)(c + 2 * wd * q));
                        t = b - c >= sc ? t >> (b - c - sc) : t << (sc - b + c);
                    }
                    const uint32_t o = (t & (((1u << (2 * wd)) - 1u) << sc)) | (first ? copy4 : copy4_2);
                    f[bb] = lds_at<uint32_t>(first ? vlut : vlut2, o);
                }
                load_row(min(J + 1, J1 - 1));  // the next group's words while this one's stores go out
                const uint32_t rowaddr = v_s + (uint32_t)((lane >> 3) * 2048 + J * 128 + (lane & 7) * 16);
#pragma unroll
                for (int bq = 0; bq < 4; ++bq)
                    stmatrix_x4_trans(rowaddr + (uint32_t)(4 * bq * 2048), f[4 * bq], f[4 * bq + 1], f[4 * bq + 2],
                                      f[4 * bq + 3]);
            }
            fence_proxy_async_smem();  // the MMA reads V through the async proxy
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(v_full);
                mbar_arrive(ring_empty(s));
            }
        }
    } else if (warp >= 8) {
        // ======================= Bs: keys and signs, thread = token =======================
        const int tau = 32 * (warp - 8) + lane;
        const float kfac = p.inv_lam_k * p.scale_log2;
        constexpr int KW = ST::KS / 4;
        // KQ: the low and high bytes of the four centroids lam_k c as fp16
        uint32_t c_lo = 0u, c_hi = 0u;
        if constexpr (KQ) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c_lo |= (p.klut[i] & 0xFFu) << (8 * i);
                c_hi |= (p.klut[i] >> 8 & 0xFFu) << (8 * i);
            }
        }
        int si = -1, Tl = 0, snt = 0;  // the tile's segment, its tile there
#pragma unroll 1
        for (int T = 0; T < ntot; ++T, ++Tl) {
#pragma unroll 1
            while (Tl >= snt) {
                snt = s_seg[++si].ntiles;
                Tl = 0;
            }
            const int s = T % kPuStages;
            bool ok = !*abort_flag && vw_wait(ring_full(s), (uint32_t)((T / kPuStages) & 1), p.err);
            if (!__all_sync(TQ_FULL_MASK, ok)) {
                *abort_flag = 1;
                break;
            }
            unsigned char* st = ring + s * SB;
            {  // the softmax's per-token factors
                const bool valid = vw_token(s_seg[si], Tl) + tau < s_seg[si].lim && ((s_held[s] >> (tau >> 4)) & 1u);
                const float kn = f16_bits_to_f32(reinterpret_cast<const uint16_t*>(st + ST::OFF_KN)[tau]);
                const uint32_t vb = reinterpret_cast<const uint16_t*>(st + ST::OFF_VN)[tau];
                const float vn = (vb & 0x7FFFu) != 0u ? f16_bits_to_f32((uint16_t)vb) : kNoNorm;
                // a row that does not see the token adds 0 times its 1 / nV, so
                // that is finite here, and a norm that is not sound goes to the
                // rows that see the token through the logit
                const bool sound = vb < 0x7C00u || vb == 0x8000u;
                float* f = reinterpret_cast<float*>(st + ST::OFF_FK) + tau;
                f[0] = valid ? (sound ? kn * kfac : nanf("")) : 0.0f;
                f[kPuTok] = valid && sound ? __log2f(vn) : 0.0f;
                f[2 * kPuTok] = valid && sound ? __frcp_rn(vn) : 0.0f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(fac_full(s));
            // S(T - NB) has read this buffer
            ok = T < NB || vw_wait(bs_free(T % NB), (uint32_t)(((T - NB) / NB) & 1), p.err);
            if (!__all_sync(TQ_FULL_MASK, ok)) {
                *abort_flag = 1;
                break;
            }
            {
                // a token past the end gets finite key values and signs of stale
                // gamma bits: its logits are masked (a select, not arithmetic)
                const uint32_t rowa = bs_buf(T) + (uint32_t)((tau >> 3) * 4096 + (tau & 7) * 16);
                const unsigned char* kr = st + ST::OFF_KC + tau * ST::KS;
                // key part: chunk c holds coordinates 8c .. 8c + 7 (four pairs)
                if constexpr (KQ) {
                    // Without a table in shared memory (random lookups there cost
                    // bank conflicts, and its bandwidth is what the kernel is short
                    // of): a nibble-aligned code is a byte permute's selector, so
                    // one permute picks the high bytes of four codes' fp16
                    // centroids, one the low bytes, and two interleave them. Word
                    // w's codes go out as 0 2 4 6 1 3 5 7 | 8 10 12 14 9 11 13 15;
                    // the query operand has the same order.
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        const uint4 k4 = reinterpret_cast<const uint4*>(kr)[half];
                        const uint32_t kw[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                        for (int wd = 0; wd < 4; ++wd) {
                            const uint32_t even = kw[wd] & 0x33333333u, odd = (kw[wd] >> 2) & 0x33333333u;
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const uint32_t se = even >> (16 * c), so = odd >> (16 * c);
                                const uint32_t he = prmt(c_hi, 0u, se), le = prmt(c_lo, 0u, se);
                                const uint32_t ho = prmt(c_hi, 0u, so), lo = prmt(c_lo, 0u, so);
                                sts128(rowa + 1024u * half + 128u * (2 * wd + c), prmt(le, he, 0x5140u), prmt(le, he, 0x7362u),
                                       prmt(lo, ho, 0x5140u), prmt(lo, ho, 0x7362u));
                            }
                        }
                    }
                } else {
                    uint32_t kw[KW + 1];
                    if constexpr (ST::KS % 16 == 0) {
#pragma unroll
                        for (int i = 0; i < KW / 4; ++i) {
                            const uint4 x = reinterpret_cast<const uint4*>(kr)[i];
                            kw[4 * i] = x.x; kw[4 * i + 1] = x.y; kw[4 * i + 2] = x.z; kw[4 * i + 3] = x.w;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < KW / 2; ++i) {
                            const uint2 x = reinterpret_cast<const uint2*>(kr)[i];
                            kw[2 * i] = x.x; kw[2 * i + 1] = x.y;
                        }
                    }
                    kw[KW] = 0u;
                    // every lookup of the row goes out before the first store
                    uint32_t x[16][4];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const bool first = !K2 || (c & 1) == 0;
                        const int wd = first ? KB : KB2;
                        const uint32_t* tab = first ? klut : klut2;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            x[c][j] = lds_at<uint32_t>(tab, field4(kw, code_bit<KB, KB2>(8 * c + 2 * j), 2 * wd));
                    }
#pragma unroll
                    for (int c = 0; c < 16; ++c) sts128(rowa + 128u * c, x[c][0], x[c][1], x[c][2], x[c][3]);
                }
                // sign part: positions 2i, 2i + 1 of sign word w hold bits i and
                // i + 16; a set bit is +gamma, a clear one -gamma
                const uint32_t gb = reinterpret_cast<const uint16_t*>(st + ST::OFF_KR)[tau];
                const uint32_t g2 = (gb | (gb << 16)) & 0x7FFF7FFFu;
#pragma unroll 1
                for (int w = 0; w < 4; ++w) {
                    const uint32_t wv = ~reinterpret_cast<const uint32_t*>(st + ST::OFF_SG + tau * 16)[w];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t y[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) y[j] = g2 ^ ((wv << (15 - (4 * c + j))) & 0x80008000u);
                        sts128(rowa + 128u * (16 + c) + 512u * w, y[0], y[1], y[2], y[3]);
                    }
                }
            }
            fence_proxy_async_smem();  // the MMA reads Bs through the async proxy
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bs_full(T % NB));
                mbar_arrive(ring_empty(s));
            }
        }
    } else {
        // ======================= softmax: two threads per query row =======================
        const int qd = warp & 3, hc = warp >> 2;  // TMEM lane quarter, column half
        const int r = 32 * qd + lane;             // query row = TMEM lane
        const uint32_t lane_base = tmem + ((uint32_t)(32 * qd) << 16);

        // The two warps of a quarter (w and w + 4, hc = 0 and 1) always take the
        // same meetings: they leave the loops at a meeting where either says so.
        asm volatile("griddepcontrol.wait;\n" ::: "memory");  // q' and u, from the query prep
        bool ok = true;    // this warp's waits
        bool left = false;  // both warps leave
#pragma unroll 1
        for (int si = 0; !left && si < nseg; ++si) {
            const VwSeg& sg = s_seg[si];
            const int ntiles = sg.ntiles, tgb = sg.tg0;
            // CTA row r is chunk token ci = (qb * 128 + r) / G and the
            // ((qb * 128 + r) % G)-th query head of KV head kv
            const int qg = sg.qb * kPuRows + r;
            const int ci = qg / G;
            const bool rok = ci < p.chunk;
            const int hj = sg.kv * G + (qg - ci * G);
            const int64_t qrow =
                rok ? ((int64_t)sg.b * p.chunk + ci) * p.hq + (p.use_table ? (int)p.head_table[hj] : hj) : -1;
            {
                // the row's window, in shared memory (registers are scarce); both
                // threads of a row write the same values, each reads its own
                const int pos = p.q_start[sg.b] + ci + 1;
                s_rows[r] = rok ? make_int2(view_low(p.view, pos), max(0, min(pos, p.lim_cap))) : make_int2(0, 0);
            }
            // ---- A of S: the hc = 0 warps write q' (column m of each limb holding
            // coordinates 2m, 2m + 1), the hc = 1 warps kappa lam_k u (column 16 w +
            // i holding sign rows 32 w + i and 32 w + i + 16). The last scores of
            // the segment before (waited for in its tile loop) are complete ----
            if (ntiles > 0) {
                const float su = p.qjl_scale / p.inv_lam_k;
                const uint32_t qlo_row = qlo_s + (uint32_t)((r >> 3) * 4096 + (r & 7) * 16);  // FL
                const float4* src = rok ? reinterpret_cast<const float4*>((hc == 0 ? p.qprime : p.u) + qrow * D) : nullptr;
#pragma unroll 1
                for (int h = 0; h < 4; ++h) {  // elements 32 h .. 32 h + 31
                    float v[32];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        // (plain loads: the launch before this one still wrote them while this one ran)
                        const float4 a = src ? src[8 * h + k] : make_float4(0.f, 0.f, 0.f, 0.f);
                        v[4 * k] = a.x; v[4 * k + 1] = a.y; v[4 * k + 2] = a.z; v[4 * k + 3] = a.w;
                    }
                    uint32_t hi[16], lo[16];
                    if (hc == 0) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            // K positions 2k, 2k + 1 (KQ: 0 2 | 4 6 | 1 3 | 5 7 of each eight)
                            const int e = KQ ? 8 * (k >> 2) + 4 * (k & 1) + ((k >> 1) & 1) : 2 * k;
                            split2(v[e], v[e + (KQ ? 2 : 1)], hi[k], lo[k]);
                        }
                        if constexpr (!FL) tmem_st16(lane_base + kVwColQlo + 16u * h, lo);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) split2(v[i] * su, v[i + 16] * su, hi[i], lo[i]);
                    }
                    if constexpr (FL) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            sts128(qlo_row + 128u * (16 * hc + 4 * h + c), lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
                    }
                    tmem_st16(lane_base + kPuColQ + 64u * hc + 16u * h, hi);
                }
                if constexpr (FL) fence_proxy_async_smem();  // the MMA reads the lo limbs through the async proxy
                tmem_st_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }

            float R = -INFINITY, Z = 0.0f;
#pragma unroll 1
            for (int T = 0; T < ntiles; ++T) {
                const int Tg = tgb + T;  // the CTA's tile count: stage and barrier phases
                const int s = Tg % kPuStages;
                ok = ok && !*abort_flag && vw_wait(fac_full(s), (uint32_t)((Tg / kPuStages) & 1), p.err) &&
                     vw_wait(s_done, (uint32_t)(Tg & 1), p.err);
                ok = __all_sync(TQ_FULL_MASK, ok);
                tc_fence_after_sync();
                // this thread's 64 columns of S (read even after a failed wait:
                // TMEM reads stay in bounds, and the values are then dropped)
                float l[64];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t x[32];
                    tmem_ld32(lane_base + kPuColS + 64u * hc + 32u * h, x);
#pragma unroll
                    for (int k = 0; k < 32; ++k) l[32 * h + k] = __uint_as_float(x[k]);
                }
                tmem_ld_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(s_empty);  // S may take the next tile's scores

                const unsigned char* st = ring + s * SB;
                const float4* fk = reinterpret_cast<const float4*>(st + ST::OFF_FK) + 16 * hc;
                // logits in log2 units, S * n_t / lam_k * scale * log2 e, and log2 nV
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float4 f = fk[k], v = fk[kPuTok / 4 + k];
                    const float2 a = __ffma2_rn(make_float2(l[4 * k], l[4 * k + 1]), make_float2(f.x, f.y), make_float2(v.x, v.y));
                    const float2 b = __ffma2_rn(make_float2(l[4 * k + 2], l[4 * k + 3]), make_float2(f.z, f.w), make_float2(v.z, v.w));
                    l[4 * k] = a.x; l[4 * k + 1] = a.y; l[4 * k + 2] = b.x; l[4 * k + 3] = b.y;
                }
                {
                    // column k (token c0 + k) is seen when it lies in [low, lim) or
                    // before the end of the sinks and lim, and its page holds it
                    const int c0 = vw_token(sg, T) + 64 * hc;
                    const int2 win = s_rows[r];
                    const int rl = win.y - c0, rw = win.x - c0, rs = p.view.sinks - c0;
                    const uint32_t held = s_held[s] >> (4 * hc) & 0xFu;
                    if (!__all_sync(TQ_FULL_MASK, rl >= 64 && (rw <= 0 || rs >= 64) && held == 0xFu)) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t two = (held >> (2 * h) & 1u) * 0xFFFFu | (held >> (2 * h + 1) & 1u) * 0xFFFF0000u;
                            const uint32_t seen = two & below(rl - 32 * h) & (~below(rw - 32 * h) | below(rs - 32 * h));
#pragma unroll
                            for (int k = 0; k < 32; ++k) l[32 * h + k] = seen >> k & 1u ? l[32 * h + k] : -INFINITY;
                        }
                    }
                }
                float mt[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) mt[k] = fmax3(l[8 * k], l[8 * k + 1], fmax3(l[8 * k + 2], l[8 * k + 3], l[8 * k + 4]));
#pragma unroll
                for (int k = 0; k < 8; ++k) mt[k] = fmax3(mt[k], l[8 * k + 5], fmax3(l[8 * k + 6], l[8 * k + 7], mt[k]));
                const float mloc = fmax3(fmax3(mt[0], mt[1], mt[2]), fmax3(mt[3], mt[4], mt[5]), fmaxf(mt[6], mt[7]));
                // both halves' maxima
                s_max[T & 1][hc][r] = mloc;
                left = pair_sync_or(1 + qd, !ok);
                if (left) break;
                // the reference (see the top): the same in both threads of the row
                const float m = fmaxf(mloc, s_max[T & 1][hc ^ 1][r]);
                float corr = 1.0f;
                if (m - 15.0f > R) {
                    const float to = m - 9.0f;
                    corr = ex2(R - to);  // the first reference: 0 of nothing
                    R = to;
                }
                const float mu = R == -INFINITY ? 0.0f : R;
                // P as fp16, tokens 64 hc + 2j, + 1 in column 32 hc + j, and what
                // it adds to Z; masked columns: 2^-inf = 0
                float2 z2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                uint32_t hi[32], lo[FL ? 32 : 1];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float4 rn = fk[kPuTok / 2 + k];
                    const float2 d0 = __fadd2_rn(make_float2(l[4 * k], l[4 * k + 1]), make_float2(-mu, -mu));
                    const float2 d1 = __fadd2_rn(make_float2(l[4 * k + 2], l[4 * k + 3]), make_float2(-mu, -mu));
                    const float2 p0 = make_float2(ex2(d0.x), ex2(d0.y)), p1 = make_float2(ex2(d1.x), ex2(d1.y));
                    z2[2 * (k & 1)] = __ffma2_rn(p0, make_float2(rn.x, rn.y), z2[2 * (k & 1)]);
                    z2[2 * (k & 1) + 1] = __ffma2_rn(p1, make_float2(rn.z, rn.w), z2[2 * (k & 1) + 1]);
                    if constexpr (FL) {
                        split2(p0.x, p0.y, hi[2 * k], lo[2 * k]);
                        split2(p1.x, p1.y, hi[2 * k + 1], lo[2 * k + 1]);
                    } else {
                        const __half2 ha = __floats2half2_rn(p0.x, p0.y), hb = __floats2half2_rn(p1.x, p1.y);
                        hi[2 * k] = *reinterpret_cast<const uint32_t*>(&ha);
                        hi[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&hb);
                    }
                }
                const float2 zz = __fadd2_rn(__fadd2_rn(z2[0], z2[1]), __fadd2_rn(z2[2], z2[3]));
                Z = fmaf(Z, corr, zz.x + zz.y);
                // P(T) and the rescale of O wait for O += P(T - 1) V(T - 1) (the
                // previous segment's last one, for a segment's first tile); a wait
                // that runs out ends both warps at their next meeting
                ok = Tg == 0 || __all_sync(TQ_FULL_MASK, vw_wait(o_done, (uint32_t)((Tg - 1) & 1), p.err));
                if (!ok) continue;
                tc_fence_after_sync();
                tmem_st32(lane_base + kVwColP + 32u * hc, hi);
                if constexpr (FL) tmem_st32(lane_base + kVwColPlo + 32u * hc, lo);
                if (T > 0 && __any_sync(TQ_FULL_MASK, corr != 1.0f)) {
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        uint32_t x[32];
                        const uint32_t a = lane_base + kPuColO + 64u * hc + 32u * h;
                        tmem_ld32(a, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float2 v = __fmul2_rn(make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])),
                                                        make_float2(corr, corr));
                            x[2 * k] = __float_as_uint(v.x);
                            x[2 * k + 1] = __float_as_uint(v.y);
                        }
                        tmem_st32(a, x);
                    }
                }
                tmem_st_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(p_full);
                    mbar_arrive(ring_empty(s));
                }
            }
            if (si == nseg - 1) asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

            // ---- this segment's partials of row r: a (rotated domain) from both
            // halves, M = R, and Z summed over the pair ----
            if (!left) {
                if (ok && ntiles > 0) ok = __all_sync(TQ_FULL_MASK, vw_wait(o_done, (uint32_t)((tgb + ntiles - 1) & 1), p.err));
                tc_fence_after_sync();
                s_max[ntiles & 1][hc][r] = Z;  // the slot that the last tile did not use
                left = pair_sync_or(1 + qd, !ok);
            }
            if (left) {  // the error word is set, the call's output is not valid
                *abort_flag = 1;
                break;
            }
            const float zsum = Z + s_max[ntiles & 1][hc ^ 1][r];
            float* out = qrow >= 0 ? p.partial + (qrow * p.n_splits + sg.slot) * (D + kPartPad) : nullptr;
            const float inv_lv = p.inv_lam_v;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                uint32_t x[32];
                tmem_ld32(lane_base + kPuColO + 64u * hc + 32u * h, x);
                tmem_ld_wait();
                if (out) {
                    float4* o4 = reinterpret_cast<float4*>(out + 64 * hc + 32 * h);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        o4[k] = ntiles == 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                                            : make_float4(__uint_as_float(x[4 * k]) * inv_lv, __uint_as_float(x[4 * k + 1]) * inv_lv,
                                                          __uint_as_float(x[4 * k + 2]) * inv_lv, __uint_as_float(x[4 * k + 3]) * inv_lv);
                }
            }
            if (out && hc == 0) {
                out[D] = zsum != zsum && R == -INFINITY ? 0.0f : R;  // all NaN is not "sees nothing", which the merge leaves out
                out[D + 1] = zsum;
            }
            // the unit's first segment also writes the slots no CTA of the unit
            // fills as empty partials (M = -inf, Z = 0, a = 0)
            if (sg.slot == 0 && qrow >= 0)
#pragma unroll 1
                for (int e = sg.nslot; e < p.n_splits; ++e) {
                    float* oe = p.partial + (qrow * p.n_splits + e) * (D + kPartPad);
#pragma unroll 1
                    for (int k = 0; k < 16; ++k) reinterpret_cast<float4*>(oe + 64 * hc)[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (hc == 0) {
                        oe[D] = -INFINITY;
                        oe[D + 1] = 0.0f;
                    }
                }
            // the pair's next write of this slot comes after both read it
            pair_sync_or(1 + qd, false);
        }  // segments
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 15) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

template <bool FL, int KB, int VB, int KB2, int VB2>
cudaError_t launch_prefill_view_t(const PrefillParams& p, cudaStream_t s) {
    auto kern = prefill_view_kernel<KB, VB, KB2, VB2, FL>;
    constexpr size_t smem = 2 * (size_t)kPuBsBytes + kPuVBytes + (size_t)kPuStages * vw_stage_bytes<PuStage<KB, VB, KB2, VB2>>();
    static_assert(smem <= 227 * 1024 - 15 * 1024, "prefill tile buffers exceed shared memory");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    // stream-K: ceil(units x unit_tiles / tiles_per_cta) CTAs
    const int64_t total = (int64_t)p.qbs * p.batch * p.hkv * p.unit_tiles;
    if (p.tiles_per_cta < 1 || p.unit_tiles < 1 || total < 1) return cudaErrorInvalidValue;
    const int64_t ctas = (total + p.tiles_per_cta - 1) / p.tiles_per_cta;
    if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
    // a programmatic dependent of the query prep: the first copies, keys and
    // values go ahead while it finishes
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kPuThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// Instantiations with 1-bit keys, and with 2-bit keys or the fractional rate.
template <bool FL>
cudaError_t prefill_view_k1(const PrefillParams& p, int vbits, cudaStream_t s) {
    switch (vbits) {
        case 1: return launch_prefill_view_t<FL, 1, 1, 1, 1>(p, s);
        case 2: return launch_prefill_view_t<FL, 1, 2, 1, 2>(p, s);
        case 3: return launch_prefill_view_t<FL, 1, 3, 1, 3>(p, s);
        case 4: return launch_prefill_view_t<FL, 1, 4, 1, 4>(p, s);
    }
    return cudaErrorInvalidValue;
}

template <bool FL>
cudaError_t prefill_view_k2(const PrefillParams& p, int vbits, bool two, cudaStream_t s) {
    switch (vbits) {
        case 1: return two ? cudaErrorInvalidValue : launch_prefill_view_t<FL, 2, 1, 2, 1>(p, s);
        case 2: return two ? launch_prefill_view_t<FL, 2, 2, 1, 1>(p, s) : launch_prefill_view_t<FL, 2, 2, 2, 2>(p, s);
        case 3: return two ? launch_prefill_view_t<FL, 2, 3, 1, 2>(p, s) : launch_prefill_view_t<FL, 2, 3, 2, 3>(p, s);
        case 4: return two ? launch_prefill_view_t<FL, 2, 4, 1, 3>(p, s) : launch_prefill_view_t<FL, 2, 4, 2, 4>(p, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace tqk
