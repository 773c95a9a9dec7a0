// paged.cuh -- the paged latent cache: page tables from request lengths, the
// append of new rows, and the work list of the attention over pages.
//
// A cache of pages is [n_pages][page][576] bf16; row j of sequence b is row
// j % page of page block_table[b][j / page].
#pragma once
#include "attn_decode.cuh"

namespace lca {

constexpr int K_TABLES = 10, K_APPEND_PAGED = 11, K_PAGED_PLAN = 12;

// ------------------------------------------------------------ scans
// Inclusive scan of one int per thread over a block, with a running
// carry for the chunks before; sums saturate at `cap` (a + b with a, b <= cap
// < 2^30 does not overflow, and min(cap, .) of sums of non-negative terms is
// associative).  Returns the exclusive sum; *total becomes the sum so far.
// Barriers inside: every thread of the block calls it.
struct BlockScan {
    int32_t wsum[32];
    int32_t carry;
};

__device__ __forceinline__ int32_t block_scan(int32_t x, int32_t cap, BlockScan &sh)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t v = min(x, cap);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v = min(v + y, cap);
    }
    if (lane == 31) sh.wsum[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int32_t w = lane < int(blockDim.x >> 5) ? sh.wsum[lane] : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off) w = min(w + y, cap);
        }
        sh.wsum[lane] = w;
    }
    __syncthreads();
    int32_t excl = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane == 0) excl = 0;
    if (warp) excl = min(excl + sh.wsum[warp - 1], cap);
    excl = min(excl + sh.carry, cap);
    const int32_t all = sh.wsum[(blockDim.x >> 5) - 1];
    __syncthreads();
    if (threadIdx.x == 0) sh.carry = min(sh.carry + all, cap);
    __syncthreads();
    return excl;
}

// ------------------------------------------------------------ page tables
// One cluster of CTAs of 128 to 1024 threads.  Every CTA scans the batch (two scans: tokens, then
// the pages they need) into shared memory; then the CTAs share the tokens and
// the new table entries out among themselves.  An entry that already stands
// in the table is only read, a new one only written (its page comes from the
// free list, not from the table), so the two passes need no order.
// seq_lens may be ctx_lens itself and taken_out may be taken: the cluster
// barrier separates every CTA's reads from the first CTA's writes.
constexpr int TB_MAX_BATCH = LCA_PAGED_MAX_BATCH;

struct TablesArgs {
    const int32_t *ctx_lens, *new_lens, *free_pages, *taken;
    int64_t n_free;
    int32_t *block_table;
    int B;
    int64_t max_blocks;
    int page_shift;
    int32_t max_tokens;
    int32_t *seq_lens, *q_start;
    int64_t *slot_map;
    int32_t *positions, *taken_out, *counts;
};

// per sequence in shared memory: first token, first new page, cached tokens
__host__ __device__ constexpr size_t tables_smem(int B) { return size_t(3 * B + 2) * 4; }

__global__ void __launch_bounds__(1024, 1) page_tables_kernel(const TablesArgs a)
{
    extern __shared__ int32_t tb_smem[];
    __shared__ BlockScan tok, pag;
    __shared__ unsigned long long asked;
    int32_t *start = tb_smem;               // [B + 1]
    int32_t *fresh = start + a.B + 1;       // [B + 1]: new pages before sequence b
    int32_t *cached = fresh + a.B + 1;      // [B]
    uint32_t rank, ranks;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    if (threadIdx.x == 0) {
        tok.carry = 0;
        pag.carry = 0;
        asked = 0;
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();

    const int32_t page = 1 << a.page_shift;
    const int64_t cap = a.max_blocks << a.page_shift;   // rows a table row can name
    const int32_t kAll = (1 << 30) - 1;
    const int64_t taken = min64(max(*a.taken, 0), a.n_free);
    for (int base = 0; base < a.B; base += int(blockDim.x)) {
        const int b = base + int(threadIdx.x);
        int32_t ctx = 0, want = 0, ask = 0;
        if (b < a.B) {
            ctx = int32_t(min64(max(a.ctx_lens[b], 0), cap));
            ask = max(a.new_lens[b], 0);
            want = int32_t(min64(ask, cap - ctx));
        }
        const int32_t t0 = block_scan(want, a.max_tokens, tok);
        const int32_t n = min(want, a.max_tokens - t0);   // tokens past max_tokens are dropped
        const int32_t len = ctx + n;
        const int32_t have = (int64_t(len) + page - 1) >> a.page_shift, old = (int64_t(ctx) + page - 1) >> a.page_shift;
        const int32_t p0 = block_scan(have - old, kAll, pag);
        unsigned long long x = ask;
#pragma unroll
        for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        if ((threadIdx.x & 31) == 0 && x) atomicAdd(&asked, x);
        if (b < a.B) {
            start[b] = t0;
            fresh[b] = p0;
            cached[b] = ctx;
        }
    }
    if (threadIdx.x == 0) {
        start[a.B] = tok.carry;
        fresh[a.B] = pag.carry;
    }
    __syncthreads();
    const int32_t T = start[a.B], P = fresh[a.B];
    if (ranks > 1) asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");

    if (rank == 0) {
        for (int b = threadIdx.x; b <= a.B; b += blockDim.x) {
            a.q_start[b] = start[b];
            if (b < a.B) a.seq_lens[b] = cached[b] + start[b + 1] - start[b];
        }
        if (threadIdx.x == 0) {
            const int32_t got = int32_t(min64(P, a.n_free - taken));
            *a.taken_out = int32_t(taken) + got;
            if (a.counts) {
                a.counts[0] = T;
                const unsigned long long lost = asked - (unsigned long long)(T);
                a.counts[1] = lost > 0x7fffffffull ? 0x7fffffff : int32_t(lost);
                a.counts[2] = got;
                a.counts[3] = P - got;
            }
        }
    }
    const int stride = int(blockDim.x * ranks);
    auto free_page = [&](int64_t k) { return taken + k < a.n_free ? a.free_pages[taken + k] : -1; };
    auto first_block = [&](int b) { return int32_t((int64_t(cached[b]) + page - 1) >> a.page_shift); };
    for (int32_t k = int32_t(rank * blockDim.x + threadIdx.x); k < P; k += stride) {
        const int b = last_le(fresh, a.B, k);
        a.block_table[size_t(b) * size_t(a.max_blocks) + first_block(b) + (k - fresh[b])] = free_page(k);
    }
    for (int64_t t = int64_t(rank * blockDim.x + threadIdx.x); t < a.max_tokens; t += stride) {
        int64_t slot = -1;
        int32_t pos = -1;
        if (t < T) {
            const int b = last_le(start, a.B, int32_t(t));
            pos = cached[b] + (int32_t(t) - start[b]);
            const int32_t k = pos >> a.page_shift, old = first_block(b);
            const int32_t pg = k < old ? a.block_table[size_t(b) * size_t(a.max_blocks) + k]
                                       : free_page(int64_t(fresh[b]) + k - old);
            if (pg >= 0) slot = (int64_t(pg) << a.page_shift) + (pos & (page - 1));
        }
        a.slot_map[t] = slot;
        if (a.positions) a.positions[t] = pos;
    }
}

// ------------------------------------------------------------ append
// rows[t] -> row slot_map[t] of the pages (a slot outside them is skipped):
// plain 16-byte copies, 72 per row, one row per 72 threads of a CTA.
constexpr int AP_ROWS = 4;                        // rows per CTA and pass
constexpr int APG_THREADS = AP_ROWS * (LCA_D * 2 / 16);

__global__ void __launch_bounds__(APG_THREADS) append_paged_kernel(const uint16_t *__restrict__ rows,
                                                                   int64_t row_pitch,
                                                                   const int64_t *__restrict__ slot_map, int64_t T,
                                                                   uint4 *__restrict__ pages, int64_t n_slots)
{
    constexpr int VEC = LCA_D * 2 / 16;
    griddep_wait();
    griddep_launch_dependents();
    const int r = threadIdx.x / VEC, v = threadIdx.x % VEC;
    for (int64_t t = int64_t(blockIdx.x) * AP_ROWS + r; t < T; t += int64_t(gridDim.x) * AP_ROWS) {
        const int64_t slot = slot_map[t];
        if (slot >= 0 && slot < n_slots)
            pages[size_t(slot) * VEC + v] = reinterpret_cast<const uint4 *>(rows + t * row_pitch)[v];
    }
}

// ------------------------------------------------------------ attention: the work list
// Every token of the batch as one item (token_rows) and its first tile in the
// batch's tile list, for batches that the attention kernel does not list
// itself.  One CTA of 128 to 1024 threads.
constexpr int PL_KEPT = 1024;

__global__ void __launch_bounds__(1024) paged_plan_kernel(const int32_t *__restrict__ seq_lens,
                                                          const int32_t *__restrict__ q_start, int B, int T,
                                                          int64_t max_rows, int32_t *__restrict__ item_seq,
                                                          int32_t *__restrict__ item_len,
                                                          int32_t *__restrict__ tile_start)
{
    __shared__ BlockScan sh;
    __shared__ int32_t starts[PL_KEPT + 1];   // q_start, for the search: a step in memory takes ~700 cycles
    if (threadIdx.x == 0) sh.carry = 0;
    griddep_wait();
    griddep_launch_dependents();
    const bool kept = B <= PL_KEPT;
    if (kept)
        for (int b = threadIdx.x; b <= B; b += int(blockDim.x)) starts[b] = q_start[b];
    const int32_t *qs = kept ? starts : q_start;
    __syncthreads();
    const int32_t kAll = 0x3fffffff;   // the host keeps the tile count below
    for (int base = 0; base < T; base += int(blockDim.x)) {
        const int t = base + int(threadIdx.x);
        int32_t len = -1;
        int b = 0;
        if (t < T) len = token_rows(qs, seq_lens, B, t, max_rows, b);
        const int32_t tiles = len > 0 ? (len + AT_TILE - 1) / AT_TILE : 0;
        const int32_t t0 = block_scan(tiles, kAll, sh);
        if (t < T) {
            item_seq[t] = b;
            item_len[t] = len;
            tile_start[t] = t0;
        }
    }
    if (threadIdx.x == 0) tile_start[T] = sh.carry;
}

}  // namespace lca
