// paged_chunk.cuh -- attention of chunks of new tokens over a paged latent
// cache: 8 tokens x 16 heads = 128 query rows per tile, on a pair of SMs.
//
// A pair of CTAs (a cluster of two) shares one tile of query rows, 64 each,
// and one stream of 64-row cache tiles.  All products are two-SM MMAs
// (cta_group::2, M = 128: 64 rows of the result in either SM) issued by one
// thread of CTA 0:
//   S [128 x 64]  = Q [128 x 576] . tile^T        N = 64: each CTA holds 32 of
//                                                 the tile's rows
//   O [128 x 512] += P [128 x 64] . tile[:, :512] two MMAs of N = 256 per 16
//                                                 rows: CTA c holds columns
//                                                 256c .. 256c+255 of all 64 rows
// Neither Q nor P nor the accumulators cross between the SMs, and a CTA
// fetches 32 whole rows and 64 half rows (68 KB) per tile for 64 query rows.
// The accumulator of 64 x 512 fp32 takes 256 columns of tensor memory, spread
// over all 128 lanes (lanes 0-63 hold rows 0-63 and the columns of the first
// half of N, lanes 64-127 the same rows and the second half), so a softmax
// thread owns half a row: 32 of the 64 logits, 256 of the 512 outputs.
//
// What bounds it: per tile and pair, 36 S steps of ~26 cycles (N = 64: the
// 64 x 16 Q operand makes shared-memory reads, 3 KB a step, the limit) and 8
// PV steps of ~66 (the tensor core's own rate), 1470 cycles for 17.8 MFLOP:
// 74% of the dense bf16 peak.  One CTA per query tile could only hold 64 rows
// (its accumulator fills half of tensor memory, S partials the rest) at half
// the S rate, ~2000 cycles for the same work on either SM; a pair with
// 128-row tiles would reach the full rate but has no shared memory left to
// hide the loads (Q 72 KB, P 16 KB, a tile's rows 72 KB and half rows 64 KB).
//
// Work: paged_chunk_plan_kernel cuts each sequence into query tiles and,
// where they are too few to fill the GPU, each tile's rows into pieces.  A
// tile in one piece writes o (as two bf16 values, hi + lo) for the W_UV
// product; pieces write (O, m, l), merged by paged_merge_kernel.
#pragma once
#include "paged.cuh"

namespace lca {

constexpr int K_CHUNK = 13, K_MERGE = 14;

constexpr int PC_TOKENS = 8;                     // per query tile
constexpr int PC_ROWS = PC_TOKENS * LCA_HEADS;   // 128 query rows per pair
constexpr int PC_TILE = 64;                      // cache rows per tile
constexpr int PC_Q = 9 * 8192;                   // 64 query rows, nine [64 x 64] blocks
constexpr int PC_K = 4 * 9 * 1024;               // 32 whole rows: [4 groups of 8][9 chunks]
constexpr int PC_V = 8 * 4 * 1024;               // 64 half rows: [8 groups][4 chunks]
constexpr int PC_P = 8192;                       // P [64 x 64] bf16
constexpr int PC_OFF_K = PC_Q;
constexpr int PC_OFF_V = PC_OFF_K + 2 * PC_K;
constexpr int PC_OFF_P = PC_OFF_V + 2 * PC_V;
constexpr int PC_OFF_X = PC_OFF_P + 2 * PC_P;    // [2][128] maxima, [128] sums
constexpr int PC_OFF_BAR = PC_OFF_X + 3 * 128 * 4;
constexpr int PC_OFF_MISC = PC_OFF_BAR + 8 * 16;
constexpr int PC_SMEM = PC_OFF_MISC + 16;
constexpr int PC_SMEM_ALLOC = PC_SMEM + 1024;
static_assert(PC_SMEM_ALLOC <= 227 * 1024, "one CTA per SM");
constexpr uint32_t PC_TM_O = 0, PC_TM_S = 256;   // O 256 columns, S two buffers of 32
constexpr int PC_THREADS = 256;
constexpr int PC_MAX_SLOTS = 160;                // partial outputs a call may write

// Per-sequence plan, and the head of it: total pieces, partial slots, split tiles.
struct ChunkPlan {
    int32_t *q0, *q1;        // [B] rows of the batch, clamped and disjoint
    int32_t *end;            // [B] tokens at or past this row index have position seq_len
    int32_t *tiles;          // [B] cache tiles of the last query tile
    int32_t *split;          // [B] pieces per query tile
    int32_t *piece_start;    // [B + 1]
    int32_t *slot_start;     // [B + 1] partial slots
    int32_t *merge_start;    // [B + 1] query tiles in several pieces
};

struct ChunkArgs {
    ChunkPlan plan;
    const int32_t *seq_lens, *q_start, *block_table;
    int B, T;
    int64_t max_blocks, n_pages;
    int page_shift;
    float sl2;
    uint16_t *o_hl;          // [T][16][2][512]
    float *part_o;           // [slots][128][512]
    float *part_ml;          // [slots][128][2]
};

// Rows that token t of sequence b attends: position + 1, within the table.
__device__ __forceinline__ int32_t chunk_rows(int32_t len, int32_t end, int32_t t, int64_t max_rows)
{
    const int64_t n = int64_t(len) - (int64_t(end) - t) + 1;
    return int32_t(n < 0 ? 0 : min64(n, max_rows));
}

// ------------------------------------------------------------ plan
// One CTA.  Offsets are read as they come: a sequence's rows are
// [q_start[b], q_start[b+1]) without those of the sequences before it
// (running maximum) and outside the batch, so the tiles number at most T.
// A piece length is tried as 1/k of the longest tile list, k = 1 .. 32 (a
// warp each): the estimate is the longest cluster's tiles, a piece costing
// kOver tiles more than its own (its queries' load, its epilogue).
__global__ void __launch_bounds__(1024) paged_chunk_plan_kernel(const ChunkArgs a, int clusters)
{
    __shared__ BlockScan sc[3];
    __shared__ int32_t wmax[32], run_max, longest;
    __shared__ float cost[32];
    __shared__ int32_t best;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        run_max = 0;
        longest = 0;
        for (int i = 0; i < 3; ++i) sc[i].carry = 0;
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const int64_t max_rows = a.max_blocks << a.page_shift;
    const ChunkPlan &p = a.plan;
    for (int base = 0; base < a.B; base += int(blockDim.x)) {
        const int b = base + int(threadIdx.x);
        int32_t lo = 0, hi = 0;
        if (b < a.B) {
            lo = min(max(a.q_start[b], 0), a.T);
            hi = min(max(a.q_start[b + 1], 0), a.T);
        }
        // running maximum of the starts, this sequence's included
        int32_t m = lo;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, m, off);
            if (lane >= off) m = max(m, y);
        }
        if (lane == 31) wmax[warp] = m;
        __syncthreads();
        if (warp == 0) {
            int32_t w = wmax[lane];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, w, off);
                if (lane >= off) w = max(w, y);
            }
            wmax[lane] = w;
        }
        __syncthreads();
        m = max(m, run_max);
        if (warp) m = max(m, wmax[warp - 1]);
        __syncthreads();
        if (threadIdx.x == 0) run_max = max(run_max, wmax[31]);
        if (b < a.B) {
            const int32_t q0 = m, q1 = max(hi, m), end = a.q_start[b + 1];
            const int32_t rows = q1 > q0 ? chunk_rows(a.seq_lens[b], end, q1 - 1, max_rows) : 0;
            const int32_t tiles = (rows + PC_TILE - 1) / PC_TILE;
            p.q0[b] = q0;
            p.q1[b] = q1;
            p.end[b] = end;
            p.tiles[b] = tiles;
            atomicMax(&longest, tiles);
        }
        __syncthreads();
    }
    // candidate k = warp + 1
    const float kOver = 4.f;
    {
        const int32_t len = max(1, (longest + warp) / (warp + 1));
        float pieces = 0.f, work = 0.f, slots = 0.f;
        for (int b = lane; b < a.B; b += 32) {
            const float nq = float((p.q1[b] - p.q0[b] + PC_TOKENS - 1) / PC_TOKENS);
            const int32_t s = max(1, (p.tiles[b] + len - 1) / len);
            pieces += nq * s;
            work += nq * p.tiles[b];
            if (s > 1) slots += nq * s;
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) {
            pieces += __shfl_xor_sync(0xffffffffu, pieces, off);
            work += __shfl_xor_sync(0xffffffffu, work, off);
            slots += __shfl_xor_sync(0xffffffffu, slots, off);
        }
        if (lane == 0) {
            const float one = float(len) + kOver, all = (work + pieces * kOver) / float(clusters);
            float c = pieces <= float(clusters) ? one : all + 0.5f * one;
            if (slots > float(PC_MAX_SLOTS) || (warp > 0 && len < 8)) c = INFINITY;
            cost[warp] = c;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int w = 0;
        for (int k = 1; k < 32; ++k)
            if (cost[k] < cost[w]) w = k;
        best = max(1, (longest + w) / (w + 1));
    }
    __syncthreads();
    const int32_t len = best, kAll = 0x3fffffff;
    for (int base = 0; base < a.B; base += int(blockDim.x)) {
        const int b = base + int(threadIdx.x);
        int32_t nq = 0, s = 1;
        if (b < a.B) {
            nq = (p.q1[b] - p.q0[b] + PC_TOKENS - 1) / PC_TOKENS;
            s = max(1, (p.tiles[b] + len - 1) / len);
            p.split[b] = s;
        }
        const int32_t x0 = block_scan(nq * s, kAll, sc[0]);
        const int32_t x1 = block_scan(s > 1 ? nq * s : 0, kAll, sc[1]);
        const int32_t x2 = block_scan(s > 1 ? nq : 0, kAll, sc[2]);
        if (b < a.B) {
            p.piece_start[b] = x0;
            p.slot_start[b] = x1;
            p.merge_start[b] = x2;
        }
    }
    if (threadIdx.x == 0) {
        p.piece_start[a.B] = sc[0].carry;
        p.slot_start[a.B] = sc[1].carry;
        p.merge_start[a.B] = sc[2].carry;
    }
}

// ------------------------------------------------------------ pair plumbing
__device__ __forceinline__ uint32_t map_to_cta(uint32_t addr, uint32_t cta)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
    return r;
}

// Arrive on a barrier of either CTA (address from map_to_cta).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// mbar_wait for barriers that threads or MMAs of the other CTA arrive on.
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, volatile int *abort, int kernel,
                                                  int site)
{
    if (mbar_try_wait_cluster(bar, parity)) return true;
    uint64_t t0 = globaltimer();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (abort && *abort) return false;
            if (globaltimer() - t0 > kWaitLimitNs) {
                report_timeout(kernel, site);
                if (abort) *abort = 1;
                return false;
            }
        }
    }
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void mma2_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on `bar` of both CTAs once every MMA this thread issued so far is done.
__device__ __forceinline__ void tc_commit_pair(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(uint16_t(3))
        : "memory");
}

// 32-byte store of eight 32-bit values.
__device__ __forceinline__ void st_global_32b(void *p, const uint32_t (&v)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// One piece of work: a query tile (rows t0 .. t0 + live - 1 of the batch) and
// the cache tiles [k0, k1) of it.
struct Piece {
    int32_t b, t0, live, len, end;
    int32_t k0, k1;
    int32_t slot;   // partial slot, or -1: the tile is in one piece
};

__device__ __forceinline__ Piece chunk_piece(const ChunkArgs &a, int32_t idx)
{
    const ChunkPlan &p = a.plan;
    Piece w;
    w.b = last_le(p.piece_start, a.B, idx);
    const int32_t q0 = p.q0[w.b], q1 = p.q1[w.b], s = p.split[w.b];
    const int32_t nq = (q1 - q0 + PC_TOKENS - 1) / PC_TOKENS, r = idx - p.piece_start[w.b];
    // the tiles with the most rows first; neighbours share their rows
    const int32_t part = r / nq, qt = nq - 1 - r % nq;
    w.t0 = q0 + PC_TOKENS * qt;
    w.live = min(PC_TOKENS, q1 - w.t0);
    w.len = a.seq_lens[w.b];
    w.end = p.end[w.b];
    const int32_t rows = chunk_rows(w.len, w.end, w.t0 + w.live - 1, a.max_blocks << a.page_shift);
    const int32_t tiles = (rows + PC_TILE - 1) / PC_TILE;
    w.k0 = int32_t(int64_t(tiles) * part / s);
    w.k1 = int32_t(int64_t(tiles) * (part + 1) / s);
    w.slot = s > 1 ? p.slot_start[w.b] + qt * s + part : -1;
    return w;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PC_THREADS, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const ChunkArgs a)
{
    extern __shared__ uint8_t pc_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(pc_smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t cta;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(cta));

    auto BAR = [&](int i) -> uint32_t { return sbase + PC_OFF_BAR + 8 * i; };
    // landed data; CTA 0's also count CTA 1's copy of the same stage
    auto kfull = [&](uint32_t n) { return BAR(int(n & 1)); };
    auto vfull = [&](uint32_t n) { return BAR(2 + int(n & 1)); };
    const uint32_t qfull = BAR(4);
    // MMAs done, in both CTAs: S(n) (so K stage n is free), PV(n) (V stage and P buffer n are)
    auto sdone = [&](uint32_t n) { return BAR(5 + int(n & 1)); };
    auto vdone = [&](uint32_t n) { return BAR(7 + int(n & 1)); };
    // CTA 0's, from the softmax warps of both: S(n) read, P(n) written, O read
    auto sread = [&](uint32_t n) { return BAR(9 + int(n & 1)); };
    auto pfull = [&](uint32_t n) { return BAR(11 + int(n & 1)); };
    const uint32_t oread = BAR(13), drain = BAR(14);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + PC_OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + PC_OFF_MISC + 4);

    if (threadIdx.x == 0) {
        const uint32_t both = cta == 0 ? 2 : 1;
        for (int s = 0; s < 2; ++s) {
            mbar_init(kfull(s), both);
            mbar_init(vfull(s), both);
            mbar_init(sdone(s), 1);
            mbar_init(vdone(s), 1);
            mbar_init(sread(s), 8);
            mbar_init(pfull(s), 8);
        }
        mbar_init(qfull, both);
        mbar_init(oread, 8);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_barrier();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_launch_dependents();
    griddep_wait();   // the plan, and everything earlier in the stream

    const int clusters = int(gridDim.x >> 1), me = int(blockIdx.x >> 1);
    const int32_t n_pieces = a.plan.piece_start[a.B];
    const int64_t no_page = a.n_pages << (a.page_shift - 3);
    const uint64_t keep = policy_evict_last();

    if (warp == 4 || warp == 5) {
        // ------------------------------------------------------------ producers
        // warp 4: the queries and this CTA's 32 whole rows of each tile;
        // warp 5: this CTA's half of the latent of all 64 rows
        const bool is_k = warp == 4;
        const int rows_per = is_k ? 32 : 64;
        const int sub_shift = min(a.page_shift, is_k ? 5 : 6);
        const int copies = rows_per >> sub_shift;
        const uint32_t bytes = is_k ? PC_K : PC_V;
        if (lane == 0) {
            prefetch_tensormap(is_k ? &map_k : &map_v);
            if (is_k) prefetch_tensormap(&map_q);
        }
        uint32_t n = 0, pieces = 0;
        bool ok = true;
        for (int32_t idx = me; idx < n_pieces && ok; idx += clusters) {
            const Piece w = chunk_piece(a, idx);
            if (w.k0 == w.k1) continue;
            if (is_k) {
                // the queries' buffer is free once the last S that read it is done
                if (n > 0) ok = mbar_wait_cluster(sdone(n - 1), ((n - 1) >> 1) & 1, abort_flag, K_CHUNK, 1);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                if (lane == 0) {
                    mbar_expect_tx(qfull, PC_Q);
                    tma_load_4d(sbase, &map_q, qfull, 0, LCA_HEADS * (w.t0 + 4 * int(cta)), 0, 0, policy_evict_first());
                }
                ++pieces;
            }
            PageWindow win;
            const int64_t first = int64_t(w.k0) * PC_TILE + (is_k ? 32 * int(cta) : 0);
            win.open(a.block_table + size_t(w.b) * size_t(a.max_blocks), first >> a.page_shift, a.max_blocks, a.n_pages,
                     lane);
            for (int32_t k = w.k0; k < w.k1; ++k, ++n) {
                const uint32_t bar = is_k ? kfull(n) : vfull(n);
                const uint32_t dst = sbase + (is_k ? PC_OFF_K + (n & 1) * PC_K : PC_OFF_V + (n & 1) * PC_V);
                ok = mbar_wait_cluster(is_k ? sdone(n) : vdone(n), ((n >> 1) & 1) ^ 1, abort_flag, K_CHUNK, 2);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                if (lane == 0) mbar_expect_tx(bar, bytes);
                const int64_t row0 = int64_t(k) * PC_TILE + (is_k ? 32 * int(cta) : 0);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c < copies) {
                        const int64_t r = row0 + (int64_t(c) << sub_shift);
                        const int32_t page = win.at(r >> a.page_shift, lane);
                        const int64_t group =
                            page >= 0 ? ((int64_t(page) << a.page_shift) + (r & ((int64_t(1) << a.page_shift) - 1))) >> 3
                                      : no_page;   // beyond the map: zeros
                        const uint32_t d = dst + ((c << sub_shift) >> 3) * (is_k ? 9 : 4) * 1024;
                        if (lane == 0)
                            tma_load_4d(d, is_k ? &map_k : &map_v, bar, 0, 0, is_k ? 0 : 4 * int(cta), int(group), keep);
                    }
                }
            }
        }
        // no copy left in flight
        if (is_k && pieces) mbar_wait(qfull, (pieces - 1) & 1, nullptr, K_CHUNK, 3);
        for (uint32_t i = n > 2 ? n - 2 : 0; i < n; ++i)
            mbar_wait(is_k ? kfull(i) : vfull(i), (i >> 1) & 1, nullptr, K_CHUNK, 4);
    } else if (warp >= 6 && cta == 1) {
        // ------------------------------------------------------------ CTA 1: tell CTA 0 what has landed here
        if (lane == 0) {
            const bool is_k = warp == 6;
            const uint32_t peer_q = map_to_cta(qfull, 0);
            uint32_t n = 0, pieces = 0;
            bool ok = true;
            for (int32_t idx = me; idx < n_pieces && ok; idx += clusters) {
                const Piece w = chunk_piece(a, idx);
                if (w.k0 == w.k1) continue;
                if (is_k) {
                    if (!(ok = mbar_wait(qfull, pieces & 1, abort_flag, K_CHUNK, 5))) break;
                    mbar_arrive_cluster(peer_q);
                    ++pieces;
                }
                for (int32_t k = w.k0; k < w.k1; ++k, ++n) {
                    const uint32_t bar = is_k ? kfull(n) : vfull(n);
                    if (!(ok = mbar_wait(bar, (n >> 1) & 1, abort_flag, K_CHUNK, 6))) break;
                    mbar_arrive_cluster(map_to_cta(bar, 0));
                }
            }
        }
    } else if (warp == 6) {
        // ------------------------------------------------------------ CTA 0: the MMAs of the pair
        if (lane == 0) {
            constexpr uint32_t IDESC_S = idesc_bf16(PC_ROWS, PC_TILE, 0, 0);
            constexpr uint32_t IDESC_PV = idesc_bf16(PC_ROWS, 256, 0, 1);
            uint32_t n = 0, pieces = 0;
            bool ok = true;
            auto issue_s = [&](uint32_t i) -> bool {
                if (!mbar_wait_cluster(kfull(i), (i >> 1) & 1, abort_flag, K_CHUNK, 7)) return false;
                if (!mbar_wait_cluster(sread(i), ((i >> 1) & 1) ^ 1, abort_flag, K_CHUNK, 8)) return false;
                tc_fence_after();
                const uint32_t kst = sbase + PC_OFF_K + (i & 1) * PC_K, d = tmem + PC_TM_S + 32 * (i & 1);
#pragma unroll 12
                for (int ks = 0; ks < 36; ++ks)
                    mma2_ss(d, sdesc_sw128(sbase + (ks >> 2) * 8192 + (ks & 3) * 32, 16, 1024),
                            sdesc_sw128(kst + (ks >> 2) * 1024 + (ks & 3) * 32, 16, 9 * 1024), IDESC_S, ks ? 1u : 0u);
                tc_commit_pair(sdone(i));
                return true;
            };
            for (int32_t idx = me; idx < n_pieces && ok; idx += clusters) {
                const Piece w = chunk_piece(a, idx);
                if (w.k0 == w.k1) continue;
                if (!(ok = mbar_wait_cluster(qfull, pieces & 1, abort_flag, K_CHUNK, 9))) break;
                if (!(ok = issue_s(n))) break;
                for (int32_t k = w.k0; k < w.k1; ++k, ++n) {
                    if (k + 1 < w.k1 && !(ok = issue_s(n + 1))) break;
                    if (k == w.k0 && !(ok = mbar_wait_cluster(oread, (pieces & 1) ^ 1, abort_flag, K_CHUNK, 10))) break;
                    if (!(ok = mbar_wait_cluster(vfull(n), (n >> 1) & 1, abort_flag, K_CHUNK, 11))) break;
                    if (!(ok = mbar_wait_cluster(pfull(n), (n >> 1) & 1, abort_flag, K_CHUNK, 12))) break;
                    tc_fence_after();
                    const uint32_t vst = sbase + PC_OFF_V + (n & 1) * PC_V, pst = sbase + PC_OFF_P + (n & 1) * PC_P;
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            mma2_ss(tmem + PC_TM_O + 128 * j, sdesc_sw128(pst + ks * 32, 16, 1024),
                                    sdesc_sw128(vst + ks * 8192 + j * 2048, 1024, 4096), IDESC_PV,
                                    (k > w.k0 || ks > 0) ? 1u : 0u);
                    tc_commit_pair(vdone(n));
                }
                ++pieces;
            }
            // no MMA left in flight (CTA 0's barrier alone: nobody else waits for it)
            asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(drain)
                         : "memory");
            mbar_wait(drain, 0, nullptr, K_CHUNK, 13);
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------ softmax and epilogue
        const int row = (32 * warp + lane) & 63, half = warp >> 1;
        const uint32_t lane_base = uint32_t(32 * warp) << 16;
        const int bar_id = 1 + (warp & 1);   // warps w and w + 2 share their rows
        float *xm = reinterpret_cast<float *>(smem + PC_OFF_X);
        const int mine = 32 * warp + lane, other = mine ^ 64;
        const int64_t max_rows = a.max_blocks << a.page_shift;
        const int tok = 4 * int(cta) + (row >> 4), head = row & 15;
        const uint32_t peer_oread = map_to_cta(oread, 0);
        uint32_t n = 0;
        bool ok = true;
        for (int32_t idx = me; idx < n_pieces && ok; idx += clusters) {
            const Piece w = chunk_piece(a, idx);
            const int32_t t = w.t0 + tok;
            const bool live = tok < w.live;
            const int32_t nv = live ? chunk_rows(w.len, w.end, t, max_rows) : 0;
            // rows that every token of the tile (of both CTAs) attends
            const int32_t nv_all = w.live == PC_TOKENS ? chunk_rows(w.len, w.end, w.t0, max_rows) : 0;
            float m = -1e30f, l = 0.f;
            PageWindow win;
            if (w.k0 < w.k1)
                win.open(a.block_table + size_t(w.b) * size_t(a.max_blocks), (int64_t(w.k0) * PC_TILE) >> a.page_shift,
                         a.max_blocks, a.n_pages, lane);
            const int sub_shift = min(a.page_shift, 6);
            for (int32_t k = w.k0; k < w.k1; ++k, ++n) {
                // which of the tile's pages are there
                uint32_t pages = 0;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c < (PC_TILE >> sub_shift) &&
                        win.at((int64_t(k) * PC_TILE + (int64_t(c) << sub_shift)) >> a.page_shift, lane) >= 0)
                        pages |= 1u << c;
                const bool whole = pages == (1u << (PC_TILE >> sub_shift)) - 1u;
                ok = mbar_wait_cluster(sdone(n), (n >> 1) & 1, abort_flag, K_CHUNK, 14);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
                float s[32];
                tmem_ld32(tmem + lane_base + PC_TM_S + 32 * (n & 1), s);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_cta(sread(n), 0));

                const int64_t row0 = int64_t(k) * PC_TILE;
                const bool edge = row0 + PC_TILE > nv_all;   // the same for both CTAs
                if (edge) {
                    // A row that is not attended by every token enters their
                    // PV product with weight 0, which a NaN or infinity in
                    // its latent would turn into NaN.  Such a row makes every
                    // logit against it non-finite: look those rows up and
                    // clear what is not finite (a token that does attend the
                    // row has the NaN in its weight already).
                    uint32_t odd = 0;
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (!(fabsf(s[x]) <= 3.4e38f)) odd |= 1u << x;
                    odd = __reduce_or_sync(0xffffffffu, odd);
                    if (odd) {
                        ok = mbar_wait_cluster(vfull(n), (n >> 1) & 1, abort_flag, K_CHUNK, 15);
                        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                        while (odd) {
                            const int r = 32 * half + __ffs(int(odd)) - 1;
                            odd &= odd - 1;
                            uint4 *p = reinterpret_cast<uint4 *>(smem + PC_OFF_V + (n & 1) * PC_V + (r >> 3) * 4096 +
                                                                 (lane >> 3) * 1024 + (r & 7) * 128 + (lane & 7) * 16);
                            const uint4 v = *p;
                            bool bad = false;
                            for (uint32_t e : {v.x, v.y, v.z, v.w})
                                bad |= (e & 0x7f80u) == 0x7f80u || (e & 0x7f800000u) == 0x7f800000u;
                            if (__any_sync(0xffffffffu, bad)) *p = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                }
                if (edge || !whole) {
                    const int64_t left = int64_t(nv) - row0 - 32 * half;
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (x >= left || !((pages >> ((32 * half + x) >> sub_shift)) & 1u)) s[x] = -INFINITY;
                }
                float tmax = s[0];
#pragma unroll
                for (int x = 1; x < 32; ++x) tmax = fmaxf(tmax, s[x]);
                xm[(n & 1) * 128 + mine] = tmax;
                named_bar_sync(bar_id, 64);
                tmax = fmaxf(tmax, xm[(n & 1) * 128 + other]) * a.sl2;
                float f = 1.f;
                if (k == w.k0) {
                    m = fmaxf(tmax, -1e30f);
                } else if (tmax > m + 8.f) {
                    f = fast_exp2(m - tmax);
                    m = tmax;
                    l *= f;
                }
                float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                    s[x] = fast_exp2(fmaf(s[x], a.sl2, -m));
                    s[x + 1] = fast_exp2(fmaf(s[x + 1], a.sl2, -m));
                    sum0 += s[x];
                    sum1 += s[x + 1];
                }
                l += sum0 + sum1;

                // P(n - 2) has been used
                ok = mbar_wait_cluster(vdone(n), ((n >> 1) & 1) ^ 1, abort_flag, K_CHUNK, 16);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                uint8_t *prow = smem + PC_OFF_P + (n & 1) * PC_P + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<uint4 *>(prow + (((4 * half + e) ^ (row & 7)) << 4)) =
                        make_uint4(pack_bf16(s[8 * e], s[8 * e + 1]), pack_bf16(s[8 * e + 2], s[8 * e + 3]),
                                   pack_bf16(s[8 * e + 4], s[8 * e + 5]), pack_bf16(s[8 * e + 6], s[8 * e + 7]));
                fence_proxy_async();
                if (__any_sync(0xffffffffu, f != 1.f)) {
                    // O must hold PV(n - 1) before it is rescaled
                    ok = mbar_wait_cluster(vdone(n - 1), ((n - 1) >> 1) & 1, abort_flag, K_CHUNK, 17);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        float o[32];
                        uint32_t r[32];
                        tmem_ld32(tmem + lane_base + PC_TM_O + 32 * c, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(o[e] * f);
                        tmem_st32(tmem + lane_base + PC_TM_O + 32 * c, r);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_cta(pfull(n), 0));
            }
            if (!ok) break;

            // ---- this thread's half row: columns 256 half .. + 255
            if (w.k0 < w.k1) {
                float *xl = xm + 256;
                xl[mine] = l;
                named_bar_sync(bar_id, 64);
                l += xl[other];
                ok = mbar_wait_cluster(vdone(n - 1), ((n - 1) >> 1) & 1, abort_flag, K_CHUNK, 18);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                tc_fence_after();
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint16_t *hl = a.o_hl + (size_t(live ? t : 0) * LCA_HEADS + head) * (2 * LCA_DC) + 256 * half;
            float *po = a.part_o + (size_t(w.slot < 0 ? 0 : w.slot) * PC_ROWS + 64 * cta + row) * LCA_DC + 256 * half;
            if (w.slot >= 0 && half == 0)
                *reinterpret_cast<float2 *>(a.part_ml + (size_t(w.slot) * PC_ROWS + 64 * cta + row) * 2) =
                    make_float2(m, l);
            if (w.slot < 0 || w.k0 < w.k1) {
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    float o[32];
                    if (w.k0 < w.k1) {
                        tmem_ld32(tmem + lane_base + PC_TM_O + 32 * c, o);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0.f;
                    }
                    if (!live) continue;
                    if (w.slot >= 0) {
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            uint32_t x[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = __float_as_uint(o[8 * v + e]);
                            st_global_32b(po + 32 * c + 8 * v, x);
                        }
                    } else {
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            uint32_t hi[8], lo[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float o0 = o[16 * v + 2 * e] * inv, o1 = o[16 * v + 2 * e + 1] * inv;
                                hi[e] = pack_bf16(o0, o1);
                                lo[e] = pack_bf16(o0 - bf_lo(hi[e]), o1 - bf_hi(hi[e]));
                            }
                            st_global_32b(hl + 32 * c + 16 * v, hi);
                            st_global_32b(hl + LCA_DC + 32 * c + 16 * v, lo);
                        }
                    }
                }
            }
            if (w.k0 < w.k1) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(peer_oread);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_barrier();   // no arrival or MMA of the pair is under way any more
    tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// ------------------------------------------------------------ merge
// Query tiles in several pieces: o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s
// per query row, one warp each (lane: 16 columns), written as hi + lo.
constexpr int MG_THREADS = 256;

__global__ void __launch_bounds__(MG_THREADS) paged_merge_kernel(const ChunkArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    const ChunkPlan &p = a.plan;
    const int warp = int(blockIdx.x) * (MG_THREADS / 32) + int(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int warps = int(gridDim.x) * (MG_THREADS / 32);
    const int32_t n = p.merge_start[a.B];
    for (int32_t i = warp; i < n * PC_ROWS; i += warps) {
        const int32_t tile = i / PC_ROWS, r = i % PC_ROWS;
        const int b = last_le(p.merge_start, a.B, tile);
        const int32_t qt = tile - p.merge_start[b], s = p.split[b];
        const int32_t t = p.q0[b] + PC_TOKENS * qt + r / LCA_HEADS;
        if (t >= p.q1[b]) continue;
        const size_t slot = size_t(p.slot_start[b] + qt * s);
        float M = -1e30f;
        for (int k = 0; k < s; ++k) M = fmaxf(M, a.part_ml[((slot + k) * PC_ROWS + r) * 2]);
        float den = 0.f, acc[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] = 0.f;
        for (int k = 0; k < s; ++k) {
            const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + ((slot + k) * PC_ROWS + r) * 2);
            if (ml.y == 0.f) continue;   // nothing attended in this piece (its O may not be there)
            const float f = fast_exp2(ml.x - M);
            den = fmaf(f, ml.y, den);
            const float4 *o = reinterpret_cast<const float4 *>(a.part_o + ((slot + k) * PC_ROWS + r) * LCA_DC + 16 * lane);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float4 x = o[v];
                acc[4 * v] = fmaf(f, x.x, acc[4 * v]);
                acc[4 * v + 1] = fmaf(f, x.y, acc[4 * v + 1]);
                acc[4 * v + 2] = fmaf(f, x.z, acc[4 * v + 2]);
                acc[4 * v + 3] = fmaf(f, x.w, acc[4 * v + 3]);
            }
        }
        const float inv = den == 0.f ? 0.f : 1.f / den;
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float o0 = acc[2 * e] * inv, o1 = acc[2 * e + 1] * inv;
            hi[e] = pack_bf16(o0, o1);
            lo[e] = pack_bf16(o0 - bf_lo(hi[e]), o1 - bf_hi(hi[e]));
        }
        uint16_t *hl = a.o_hl + (size_t(t) * LCA_HEADS + r % LCA_HEADS) * (2 * LCA_DC) + 16 * lane;
        st_global_32b(hl, hi);
        st_global_32b(hl + LCA_DC, lo);
    }
}

}  // namespace lca
