// paged_chunk.cuh -- attention of chunks of new tokens over a paged latent
// cache: 8 tokens x 16 heads = 128 query rows per query tile, on a pair of SMs.
//
// A pair of CTAs (a cluster of two) shares one query tile, 64 query rows each,
// and one stream of 128-row cache tiles.  All products are two-SM MMAs
// (cta_group::2, M = 128: 64 rows of the result in either SM), issued by CTA 0:
//   S [128 x 128] = Q [128 x 576] . tile^T        each CTA holds 64 of the
//                                                 tile's rows
//   O [128 x 512] += P [128 x 128] . tile[:, :512] two MMAs of N = 256 per 16
//                                                 rows: CTA c holds columns
//                                                 256c .. 256c+255 of all rows
// Neither Q nor P nor the accumulators cross between the SMs.  The accumulator
// of 64 x 512 fp32 takes 256 columns of tensor memory, spread over all 128
// lanes (lanes 0-63 hold rows 0-63 and the columns of the first half of N,
// lanes 64-127 the same rows and the second half), so a softmax thread owns
// half a row: 64 of the 128 logits, 256 of the 512 outputs.
//
// A tile is fetched in slots of 8 KB: nine for S ([64 rows][64 columns], this
// CTA's rows) and eight for PV ([16 rows][256 columns], this CTA's columns),
// each freed by the commit of the MMAs that read it.  S and PV have a ring of
// slots each (one tile's): only where one warp uses and frees a ring's slots in
// order does the parity of a slot's barrier tell two of its uses apart.
//
// Online softmax: per query row a reference m, raised (and O rescaled) only
// when the maximum grows by more than 2^8; the weights 2^(z - m) enter PV as
// bf16 (off by 2^-8 at most, the operand's type), their sum l is of the fp32
// values.  o = O / l leaves as two bf16 values, hi + lo (off by 2^-16), for the
// W_UV product of paged_wuv.cuh.
//
// What bounds it: per cache tile and pair 36 S steps of 34 cycles and 16 PV
// steps of 66, 2270 cycles of tensor core for 17.8 MFLOP a CTA (96% of the
// dense peak; M = 256 would leave no tensor memory for S, tiles of 64 rows
// would double the reads of Q, 2950 cycles).  Measured, 2048 tokens over 32768
// rows: 3000 cycles a tile, 1.62 ms for the kernel, 1.40 PFLOP/s, tensor pipe
// active 75%, at the power cap's 1.6 GHz; 1.9 ms a call back to back.  What
// holds the rest is the chain from a tile's S through softmax, P and PV to the
// next P (there is room for one P beside the rings): without any product or
// copy the same loops take 1.1 ms.
// With few tokens a sequence the rows come from memory: 16 x 2..5 tokens over
// 138515 rows, 160 MB, 47 us, of which 8 are the first tile's way through.
//
// Work: paged_chunk_plan_kernel lays the query tiles' cache tiles end to end
// and cuts them into one equal range per pair; a query tile that a border cuts
// leaves partial (O, m, l) per piece, merged in order by paged_merge_kernel.
#pragma once
#include <type_traits>

#include "paged.cuh"

namespace lca {

constexpr int K_CHUNK = 13, K_MERGE = 14;

constexpr int PC_TOKENS = 8;                     // per query tile
constexpr int PC_ROWS = PC_TOKENS * LCA_HEADS;   // 128 query rows per pair
constexpr int PC_TILE = 128;                     // cache rows per tile
constexpr int PC_Q = 9 * 8192;                   // 64 query rows, nine [64 x 64] blocks
constexpr int PC_SLOT = 8192;
constexpr int PC_KS = 9, PC_VS = 8;              // slots of a tile: for S, for PV
constexpr int PC_KRING = 9, PC_VRING = 8;        // (a tile's PV slots fit the ring: see vready)
constexpr int PC_SLOTS = PC_KRING + PC_VRING;
constexpr int PC_P = 2 * 8192;                   // P [64 x 128] bf16, two [64 x 64] blocks
constexpr int PC_OFF_P = PC_Q;
constexpr int PC_OFF_RING = PC_OFF_P + PC_P;
constexpr int PC_OFF_X = PC_OFF_RING + PC_SLOTS * PC_SLOT;   // [2][128] row maxima or sums
constexpr int PC_OFF_BAR = PC_OFF_X + 2 * 128 * 4;
constexpr int PC_BARS = 2 * PC_SLOTS + 13;
constexpr int PC_OFF_MISC = PC_OFF_BAR + 8 * PC_BARS;
constexpr int PC_SMEM = PC_OFF_MISC + 16;
constexpr int PC_SMEM_ALLOC = PC_SMEM + 1024;
static_assert(PC_SMEM_ALLOC <= 227 * 1024, "one CTA per SM");
constexpr uint32_t PC_TM_O = 0, PC_TM_S = 256;   // O 256 columns, S two buffers of 64
constexpr int PC_SOFTMAX = 4;                    // warps 0 .. 3
constexpr int PC_KWARPS = 3, PC_VWARPS = 2;      // fetch: warps 4 .. 6 for S, 7, 8 for PV
constexpr int PC_WARP_S = 9, PC_WARP_PV = 10;    // MMA issue (CTA 0)
constexpr int PC_THREADS = 32 * 11;
constexpr int PC_MAX_CLUSTERS = 80;              // partial outputs: two per cluster
constexpr int PC_MIN_UNITS = 3;                  // fewer clusters rather than shorter ranges: every piece is
                                                 // one more to merge
constexpr int PC_PLAN_KEPT = 1024;               // sequences, and query tiles, that the plan keeps in shared memory
constexpr int PC_OVER = 4;                       // cost of a piece beyond its tiles, in tiles.  A piece of n tiles
                                                 // takes about 5.2 + 1.65 n us, which says 3.2; taken by
                                                 // measurement instead: with 2, 3, 4, 5 four prompts of 611 ..
                                                 // 1733 tokens take 255, 246, 241, 241 us, 16 x 2..5 tokens 65.3,
                                                 // 65.8, 66.0, 66.3, a mixed batch 176.5, 176, 175, 175.5

// A query tile: tokens t0 .. t0 + live - 1 of sequence b; token t attends
// row_base + t rows (within the table).  The work of all query tiles is laid
// end to end in units of one cache tile, PC_OVER more for each query tile,
// and cut into one equal range per cluster.
struct alignas(16) ChunkTile {
    int32_t b, t0, live, tiles;
    int64_t row_base, unit0;
};

// A query tile that a cluster's border cuts: pieces by the clusters c0 .. c1.
struct alignas(16) ChunkMerge {
    int32_t t0, live, c0, c1;
};

struct ChunkPlan {
    int32_t *q0, *q1;        // [B] rows of the batch, clamped and disjoint (batches above PC_PLAN_KEPT)
    int32_t *tile0;          // [B] first query tile (likewise)
    ChunkTile *tile;         // [T / 8 + B + 1]; tile[nq].unit0: all units
    int32_t *first;          // [PC_MAX_CLUSTERS] query tile of the cluster's first unit
    int32_t *nq;             // [2] query tiles, clusters with work
    ChunkMerge *merge;       // [PC_MAX_CLUSTERS] by the first border inside; c1 < 0: none
};

struct ChunkArgs {
    ChunkPlan plan;
    const int32_t *seq_lens, *q_start, *block_table;
    int B, T;
    int64_t max_blocks, n_pages;
    int page_shift;
    float sl2;
    uint16_t *o_hl;          // [T][16][2][512]
    float *part_o;           // [2 * clusters][128][512]
    float *part_ml;          // [2 * clusters][128][2]
};

__device__ __forceinline__ int32_t clamp_rows(int64_t n, int64_t max_rows)
{
    return int32_t(n < 0 ? 0 : min64(n, max_rows));
}

// ------------------------------------------------------------ plan
// Exclusive sum over the block plus the carry (see block_scan).
struct BlockScan64 {
    int64_t wsum[32];
    int64_t carry;
};

__device__ __forceinline__ int64_t block_scan64(int64_t x, BlockScan64 &sh)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = int(blockDim.x >> 5);
    int64_t v = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += y;
    }
    if (lane == 31) sh.wsum[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int64_t w = lane < warps ? sh.wsum[lane] : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off) w += y;
        }
        sh.wsum[lane] = w;
    }
    __syncthreads();
    const int64_t excl = v - x + (warp ? sh.wsum[warp - 1] : 0) + sh.carry;
    const int64_t all = sh.wsum[warps - 1];
    __syncthreads();
    if (threadIdx.x == 0) sh.carry += all;
    __syncthreads();
    return excl;
}

// One CTA.  Offsets are read as they come: a sequence's rows are
// [q_start[b], q_start[b+1]) without those of the sequences before it
// (running maximum) and outside the batch, so the query tiles number at most
// T / 8 + B.  128 to 1024 threads.
__global__ void __launch_bounds__(1024) paged_chunk_plan_kernel(const ChunkArgs a, int clusters)
{
    __shared__ BlockScan sc;
    __shared__ BlockScan64 sc64;
    __shared__ int32_t wmax[32], run_max, sq0[PC_PLAN_KEPT], sq1[PC_PLAN_KEPT], st0[PC_PLAN_KEPT];
    __shared__ int64_t su0[PC_PLAN_KEPT + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        run_max = 0;
        sc.carry = 0;
        sc64.carry = 0;
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const int64_t max_rows = a.max_blocks << a.page_shift;
    const ChunkPlan &p = a.plan;
    const bool small = a.B <= PC_PLAN_KEPT;
    int32_t *q0s = small ? sq0 : p.q0, *q1s = small ? sq1 : p.q1, *tile0 = small ? st0 : p.tile0;
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
            int32_t w = lane < int(blockDim.x >> 5) ? wmax[lane] : 0;
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
        if (threadIdx.x == 0) run_max = max(run_max, wmax[(blockDim.x >> 5) - 1]);
        const int32_t q0 = m, q1 = max(hi, m);
        const int32_t t0 = block_scan(b < a.B ? (q1 - q0 + PC_TOKENS - 1) / PC_TOKENS : 0, 0x3fffffff, sc);
        if (b < a.B) {
            q0s[b] = q0;
            q1s[b] = q1;
            tile0[b] = t0;
        }
    }
    __syncthreads();   // every sequence's entries are written
    const int32_t nq = sc.carry;
    for (int base = 0; base < nq; base += int(blockDim.x)) {
        const int i = base + int(threadIdx.x);
        ChunkTile w{};
        if (i < nq) {
            w.b = last_le(tile0, a.B, i);
            const int32_t q0 = q0s[w.b], q1 = q1s[w.b];
            // the tiles with the most rows first
            w.t0 = q0 + PC_TOKENS * ((q1 - q0 + PC_TOKENS - 1) / PC_TOKENS - 1 - (i - tile0[w.b]));
            w.live = min(PC_TOKENS, q1 - w.t0);
            w.row_base = int64_t(a.seq_lens[w.b]) - a.q_start[w.b + 1] + 1;
            w.tiles = (int64_t(clamp_rows(w.row_base + w.t0 + w.live - 1, max_rows)) + PC_TILE - 1) / PC_TILE;
        }
        w.unit0 = block_scan64(i < nq ? w.tiles + PC_OVER : 0, sc64);
        if (i < nq) {
            p.tile[i] = w;
            if (i < PC_PLAN_KEPT) su0[i] = w.unit0;
        }
    }
    const int64_t units = sc64.carry;
    const int active = int(min64(clusters, (units + PC_MIN_UNITS - 1) / PC_MIN_UNITS));
    if (threadIdx.x == 0) {
        p.tile[nq].unit0 = units;
        p.nq[0] = nq;
        p.nq[1] = active;
    }
    __syncthreads();
    // Cluster c starts at unit c * units / active: its query tile, and whether
    // that border cuts the tile's cache tiles.
    __shared__ int32_t at_tile[PC_MAX_CLUSTERS];
    __shared__ bool cuts[PC_MAX_CLUSTERS];
    const auto unit0 = [&](int i) { return nq <= PC_PLAN_KEPT ? su0[i] : p.tile[i].unit0; };
    const int c = threadIdx.x;
    if (c < active) {
        const int64_t at = split_begin(c, units, active);
        int lo = 0, hi = nq - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (unit0(mid) <= at) lo = mid;
            else hi = mid - 1;
        }
        p.first[c] = lo;
        at_tile[c] = lo;
        cuts[c] = at > unit0(lo) + PC_OVER;
    }
    __syncthreads();
    if (c < clusters) {
        ChunkMerge g{0, 0, 0, -1};
        if (c > 0 && c < active && cuts[c] && !(cuts[c - 1] && at_tile[c - 1] == at_tile[c])) {
            g = ChunkMerge{p.tile[at_tile[c]].t0, p.tile[at_tile[c]].live, c - 1, c};
            while (g.c1 + 1 < active && cuts[g.c1 + 1] && at_tile[g.c1 + 1] == at_tile[c]) ++g.c1;
        }
        p.merge[c] = g;
    }
}

// ------------------------------------------------------------ pair plumbing
__device__ __forceinline__ uint32_t map_to_cta(uint32_t addr, uint32_t cta)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
    return r;
}

// Arrive on a barrier of either CTA (address from map_to_cta).  What it
// announces is read where it was written, by the MMAs of the announcing SM (P,
// tensor memory) after the proxy or tcgen05 fence in front; a release at
// cluster scope would wait ~900 cycles for this thread's global stores.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One lane of the (converged) warp, the same each time.  MMAs issued under it
// take 26 to 37 cycles each (80 under `lane == 0`).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.b32 %0, 1, 0, P;\n\t}" : "=r"(p));
    return p != 0;
}

// mbar_try_wait without its wait.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// One lane looks at a barrier for the whole warp (32 lanes that poll take the
// shared-memory pipe from everybody else); the same answer in every lane.  The
// look is predicated, not branched to: a warp whose lanes parted in a wait
// stayed parted through the tile that followed and ran it twice.
__device__ __forceinline__ bool warp_try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred E, Q;\n\t"
        "elect.sync _|E, 0xffffffff;\n\t"
        "setp.ne.b32 Q, 0, 0;\n\t"
        "@E mbarrier.try_wait.parity.shared::cta.b64 Q, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, Q;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return __any_sync(0xffffffffu, ok);
}

// The loop stands apart: with it inline at every wait and the loops over slots
// unrolled, the warps' roles kept evicting each other's instructions.  The
// clock is read only after many looks: a read of %globaltimer takes long.
__device__ __noinline__ bool warp_wait_more(uint32_t bar, uint32_t parity, volatile int *abort, int site)
{
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (warp_try_wait(bar, parity)) return true;
        if ((it & 255u) == 0) {
            if (__any_sync(0xffffffffu, *abort != 0)) return false;
            const uint64_t t = __shfl_sync(0xffffffffu, globaltimer(), 0);
            if (t0 == 0) t0 = t;
            if (t - t0 > kWaitLimitNs) {
                report_timeout(K_CHUNK, site);
                *abort = 1;
                return false;
            }
        }
    }
}

// The same for one thread.
__device__ __noinline__ bool wait_more(uint32_t bar, uint32_t parity, volatile int *abort, int site)
{
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 255u) == 0) {
            if (*abort) return false;
            const uint64_t t = globaltimer();
            if (t0 == 0) t0 = t;
            if (t - t0 > kWaitLimitNs) {
                report_timeout(K_CHUNK, site);
                *abort = 1;
                return false;
            }
        }
    }
}

// mbar_wait by a whole, converged warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort, int site)
{
    const bool ok = warp_try_wait(bar, parity) || warp_wait_more(bar, parity, abort, site);
    __syncwarp();
    return ok;
}

// A place in a ring of N slots: its slot, and the parity of its use.
template <int N>
struct RingPlace {
    uint32_t slot = 0, par = 0;
    __device__ __forceinline__ void operator++()
    {
        if (++slot == N) {
            slot = 0;
            par ^= 1;
        }
    }
    __device__ __forceinline__ void skip(uint32_t n)   // n <= N
    {
        slot += n;
        if (slot >= N) {
            slot -= N;
            par ^= 1;
        }
    }
    // Each lane looks at a place of its own, `ahead` and more places on (barriers
    // from `first` on): one look, of ~100 cycles, serves several slots.
    __device__ __forceinline__ bool look(uint32_t first, int ahead, int lane) const
    {
        uint32_t s = slot + uint32_t(ahead + lane), q = par;
        if (s >= N) {
            s -= N;
            q ^= 1;
        }
        return ahead + lane < N && mbar_test(first + 8 * s, q);
    }
    // How many places in a row were complete in a look; if none is, waits for the
    // next one.  0: given up.
    __device__ __forceinline__ int count(uint32_t first, bool looked, volatile int *abort, int site) const
    {
        const uint32_t there = __ballot_sync(0xffffffffu, looked);
        if (there & 1u) return __ffs(int(~there)) - 1;
        return warp_wait(first + 8 * slot, par, abort, site) ? 1 : 0;
    }
};

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

// 4-D tiled TMA load into this CTA, its bytes counted on a barrier of either
// CTA of the pair (address from map_to_cta).
__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z,
                                                 int w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// Pairs of fp32 values: two multiply-adds or adds in one instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Power of two that brings a reference m of 2^30 and more below 2^30 (1 below
// that).  A weight's exponent z - m is one multiply-add of the logit, so it holds
// what m was rounded by, up to 2^-24 |m|: a factor that all of a row's weights
// share, but none that fp32 holds where m reaches 2^31 (the weights were all
// infinite or zero there).  Shrunk, it is 2^32 at most, and logits that differ in
// fp32 are still 2^5 or more apart: the weights stay one-hot.
__device__ __forceinline__ float shrink_of(float m)
{
    const uint32_t e = __float_as_uint(m) & 0x7f800000u;
    return __uint_as_float(min((283u << 23) - e, 127u << 23));
}

// A cluster's pieces: query tile q and the cache tiles [k0, k1) of it.
struct ChunkPiece {
    ChunkTile t;
    int32_t k0, k1;
    int32_t slot;   // partial slot, or -1: the query tile is in one piece
    __device__ __forceinline__ int32_t n() const { return k1 - k0; }
    // PV slots of the piece's i-th cache tile (16 rows each; rows past the last are left out)
    __device__ __forceinline__ int32_t v_slots(int i, int64_t max_rows) const
    {
        if (k0 + i + 1 < t.tiles) return PC_VS;
        const int32_t rows = clamp_rows(t.row_base + t.t0 + t.live - 1, max_rows);
        return (rows - (t.tiles - 1) * PC_TILE + 15) >> 4;
    }
};

struct ChunkRange {
    int32_t q, nq, cluster;
    int64_t begin, end;
    __device__ __forceinline__ ChunkRange(const ChunkPlan &p, int c)
    {
        nq = p.nq[0];
        const int active = p.nq[1];
        cluster = c;
        q = nq;
        begin = end = 0;
        if (c < active) {
            const int64_t units = p.tile[nq].unit0;
            begin = split_begin(c, units, active);
            end = split_begin(c + 1, units, active);
            q = p.first[c];
        }
    }
    // the next piece with cache tiles, or of a query tile that has none
    __device__ __forceinline__ bool next(const ChunkPlan &p, ChunkPiece &w)
    {
        for (; q < nq; ++q) {
            w.t = p.tile[q];
            if (w.t.unit0 >= end) break;
            const int64_t u = w.t.unit0 + PC_OVER;
            w.k0 = clamp_rows(begin - u, w.t.tiles);
            w.k1 = clamp_rows(end - u, w.t.tiles);
            w.slot = w.n() == w.t.tiles ? -1 : 2 * cluster + (w.k0 == 0 ? 1 : 0);
            if (w.n() > 0 || (w.t.tiles == 0 && w.t.unit0 >= begin)) {
                ++q;
                return true;
            }
        }
        return false;
    }
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PC_THREADS, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const ChunkArgs a)
{
    extern __shared__ uint8_t pc_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(pc_smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    uint32_t cta;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(cta));

    auto BAR = [&](int i) -> uint32_t { return sbase + PC_OFF_BAR + 8 * i; };
    // CTA 0's: both CTAs' copies into a slot have landed / its own: the slot is free.
    auto kfull = [&](uint32_t slot) { return BAR(int(slot)); };
    auto kempty = [&](uint32_t slot) { return BAR(PC_KRING + int(slot)); };
    auto vfull = [&](uint32_t slot) { return BAR(2 * PC_KRING + int(slot)); };
    auto vempty = [&](uint32_t slot) { return BAR(2 * PC_KRING + PC_VRING + int(slot)); };
    auto kaddr = [&](uint32_t slot) { return sbase + PC_OFF_RING + slot * PC_SLOT; };
    auto vaddr = [&](uint32_t slot) { return sbase + PC_OFF_RING + (PC_KRING + slot) * PC_SLOT; };
    constexpr int B0 = 2 * PC_SLOTS;
    const uint32_t qfull = BAR(B0);
    // MMAs done, in both CTAs: S(n), PV(n)
    auto sdone = [&](uint32_t n) { return BAR(B0 + 1 + int(n & 1)); };
    auto vdone = [&](uint32_t n) { return BAR(B0 + 3 + int(n & 1)); };
    // CTA 0's, from the softmax warps of both: S(n) read, P(n) written, O read
    auto sread = [&](uint32_t n) { return BAR(B0 + 5 + int(n & 1)); };
    auto pfull = [&](uint32_t n) { return BAR(B0 + 7 + int(n & 1)); };
    const uint32_t oread = BAR(B0 + 9);
    const uint32_t vready = BAR(B0 + 10);   // in both CTAs: an edge tile's PV slots have landed
    const uint32_t drain_s = BAR(B0 + 11), drain_pv = BAR(B0 + 12);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + PC_OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + PC_OFF_MISC + 4);

    if (threadIdx.x == 0) {
        for (int i = 0; i < PC_BARS; ++i) mbar_init(BAR(i), i < B0 + 5 ? 1 : i <= B0 + 9 ? 2 * PC_SOFTMAX : 1);
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

    const int64_t max_rows = a.max_blocks << a.page_shift;
    ChunkRange range(a.plan, int(blockIdx.x >> 1));
    ChunkPiece w;

    // ---------------------------------------------------------------- producers
    // One thread each; producer p of STEP brings a ring's uses p, p + STEP, ...
    // (wait, expect and copy take it ~400 cycles a slot; the MMAs use a slot of
    // either ring every 330).  STEP < ring, so a producer has seen the use before
    // last of its next slot freed.
    const auto produce = [&](auto is_k_, uint32_t p) {
        constexpr bool K = decltype(is_k_)::value;
        constexpr uint32_t RING = K ? PC_KRING : PC_VRING, STEP = K ? PC_KWARPS : PC_VWARPS;
        static_assert(STEP < RING && PC_KS % PC_KWARPS == 0 && PC_VS % PC_VWARPS == 0, "slots per tile and producer");
        const uint32_t full0 = K ? kfull(0) : vfull(0), empty0 = K ? kempty(0) : vempty(0);
        const uint32_t slot0 = K ? kaddr(0) : vaddr(0), full_pair = map_to_cta(full0, 0);
        // rows, pages and 8-row groups are below 2^31
        const int shift = a.page_shift, in_page = (1 << shift) - 1, blocks = int(a.max_blocks), pages = int(a.n_pages);
        const int no_page = pages << (shift - 3);   // beyond the map: zeros
        prefetch_tensormap(K ? &map_k : &map_v);
        if (K && p == 0) prefetch_tensormap(&map_q);
        uint32_t n = 0, x = p, base = 0;   // tiles; this producer's next use of the ring; the tile's first use
        uint32_t slot = p, par = 1;        // x's slot, and the parity that says that it is free
        bool ok = true;
        const auto take = [&]() {
            if (!mbar_try_wait(empty0 + 8 * slot, par)) ok = wait_more(empty0 + 8 * slot, par, abort_flag, 2);
            if (ok && cta == 0) mbar_expect_tx(full0 + 8 * slot, 2 * PC_SLOT);   // both CTAs' bytes
            return ok;
        };
        const auto step = [&]() {
            x += STEP;
            slot += STEP;
            if (slot >= RING) {
                slot -= RING;
                par ^= 1;
            }
        };
        while (ok && range.next(a.plan, w)) {
            if (w.n() == 0) continue;
            if (K && p == 0) {
                // the queries' buffer is free once the last S that read it is done
                if (n > 0) ok = wait_more(sdone(n - 1), ((n - 1) >> 1) & 1, abort_flag, 1);
                if (!ok) break;
                if (cta == 0) mbar_expect_tx(qfull, 2 * PC_Q);
                tma_load_4d_pair(sbase, &map_q, map_to_cta(qfull, 0), 0, LCA_HEADS * (w.t.t0 + 4 * int(cta)), 0, 0);
            }
            const int32_t *table = a.block_table + size_t(w.t.b) * size_t(a.max_blocks);
            // (an entry is looked at only when it is used, a tile later: no wait for the load)
            const auto page_of = [&](int r) { return (r >> shift) < blocks ? __ldg(table + (r >> shift)) : -1; };
            const auto group_of = [&](int page, int r) {
                return uint32_t(page) < uint32_t(pages) ? (page << (shift - 3)) + ((r & in_page) >> 3) : no_page;
            };
            // The rows that this producer brings of a tile lie in up to four
            // pages; those of the next tile are looked up a tile ahead.  K: all 64
            // rows in steps of `sub`; V: the 16 rows of each of its parts.
            const int sub = K ? min(64, 1 << shift) : 16 * int(STEP);
            constexpr int LOOKUPS = K ? 4 : PC_VS / PC_VWARPS;
            int row0 = w.k0 * PC_TILE + (K ? 64 * int(cta) : 16 * int(x - base));
            int page[LOOKUPS], group[LOOKUPS];
#pragma unroll
            for (int c = 0; c < LOOKUPS; ++c) page[c] = !K || c * sub < 64 ? page_of(row0 + c * sub) : -1;
            const int last = w.v_slots(w.n() - 1, max_rows);
            for (int i = w.n(); i > 0 && ok; --i, ++n, row0 += PC_TILE) {
#pragma unroll
                for (int c = 0; c < LOOKUPS; ++c) group[c] = group_of(page[c], row0 + c * sub);
#pragma unroll
                for (int c = 0; c < LOOKUPS; ++c)
                    if (i > 1 && (!K || c * sub < 64)) page[c] = page_of(row0 + PC_TILE + c * sub);
                if (K) {
                    if (sub == 64) {
#pragma unroll
                        for (int c = 0; c < PC_KS / PC_KWARPS; ++c, step())
                            if (ok && take())
                                tma_load_4d_pair(slot0 + slot * PC_SLOT, &map_k, full_pair + 8 * slot, 0, 0,
                                                 int(p) + PC_KWARPS * c, group[0]);
                    } else {
#pragma unroll 1
                        for (int c = 0; c < PC_KS / PC_KWARPS; ++c, step()) {
                            if (!ok || !take()) continue;
                            const int part = int(p) + PC_KWARPS * c;
                            const uint32_t dst = slot0 + slot * PC_SLOT, bar = full_pair + 8 * slot;
                            tma_load_4d_pair(dst, &map_k, bar, 0, 0, part, group[0]);
                            tma_load_4d_pair(dst + sub * 128, &map_k, bar, 0, 0, part, group[1]);
                            if (sub == 16) {
                                tma_load_4d_pair(dst + 4096, &map_k, bar, 0, 0, part, group[2]);
                                tma_load_4d_pair(dst + 6144, &map_k, bar, 0, 0, part, group[3]);
                            }
                        }
                    }
                    base += PC_KS;
                } else {
                    const uint32_t end = base + uint32_t(i > 1 ? PC_VS : last);
#pragma unroll
                    for (int c = 0; c < LOOKUPS; ++c)
                        if (ok && x < end && take()) {
                            tma_load_4d_pair(slot0 + slot * PC_SLOT, &map_v, full_pair + 8 * slot, 0, 0, 4 * int(cta),
                                             group[c]);
                            step();
                        }
                    base = end;
                }
            }
        }
        // No copy left in flight, and every commit that arrives at this CTA
        // has: this producer's among the ring's last uses, backwards.
        while (ok && x >= STEP && x - STEP + RING >= base) {
            x -= STEP;
            if (slot < STEP) {
                slot += RING;
                par ^= 1;
            }
            slot -= STEP;
            if (cta == 0) ok = wait_more(full0 + 8 * slot, par ^ 1, abort_flag, 4);
            ok = ok && wait_more(empty0 + 8 * slot, par ^ 1, abort_flag, 6);
        }
        if (!ok) {   // given up: copies may still be under way
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 10000000ull) __nanosleep(1000);
        }
    };

    if (warp >= PC_SOFTMAX && warp < PC_SOFTMAX + PC_KWARPS) {
        if (lane == 0) produce(std::true_type{}, uint32_t(warp - PC_SOFTMAX));
        __syncwarp();
    } else if (warp >= PC_SOFTMAX + PC_KWARPS && warp < PC_WARP_S) {
        if (lane == 0) produce(std::false_type{}, uint32_t(warp - PC_SOFTMAX - PC_KWARPS));
        __syncwarp();
    } else if (warp == PC_WARP_S && cta == 0) {
        // ------------------------------------------------------------ S = Q . tile^T for the pair
        constexpr uint32_t IDESC_S = idesc_bf16(PC_ROWS, PC_TILE, 0, 0);
        const uint64_t q_desc = sdesc_sw128(sbase, 16, 1024), k_desc = sdesc_sw128(kaddr(0), 16, 1024);
        // chunks c .. c + count - 1 of a tile, from slot `at` on
        const auto s_mmas = [&](RingPlace<PC_KRING> at, uint32_t d, int c, int count) {
            uint64_t qd = q_desc + uint64_t(c * (8192 >> 4));
#pragma unroll 1
            for (; count > 0; --count, ++c, ++at, qd += 8192 >> 4) {
                const uint64_t kd = k_desc + uint64_t(at.slot * (PC_SLOT >> 4));
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma2_ss(d, qd + 2 * ks, kd + 2 * ks, IDESC_S, c + ks ? 1u : 0u);
                tc_commit_pair(kempty(at.slot));
            }
        };
        RingPlace<PC_KRING> at;
        uint32_t n = 0, pieces = 0;
        bool ok = true;
        while (ok && range.next(a.plan, w)) {
            const int m = __shfl_sync(0xffffffffu, w.n(), 0);
            if (m == 0) continue;
            if (!(ok = warp_wait(qfull, pieces & 1, abort_flag, 8))) break;
            for (int i = 0; i < m && ok; ++i, ++n) {
                if (!(ok = warp_wait(sread(n), ((n >> 1) & 1) ^ 1, abort_flag, 9))) break;
                const uint32_t d = tmem + PC_TM_S + 64 * (n & 1);
                bool looked = at.look(kfull(0), 0, lane);
                for (int c = 0; c < PC_KS;) {
                    const int got = min(at.count(kfull(0), looked, abort_flag, 10), PC_KS - c);
                    if (!(ok = got > 0)) break;
                    tc_fence_after();
                    if (got > 1 && elect_one()) s_mmas(at, d, c, got - 1);
                    __syncwarp();
                    c += got - 1;
                    at.skip(uint32_t(got - 1));
                    looked = at.look(kfull(0), 1, lane);   // comes back while the last one's MMAs are issued
                    if (elect_one()) {
                        s_mmas(at, d, c, 1);
                        if (c + 1 == PC_KS) tc_commit_pair(sdone(n));
                    }
                    __syncwarp();
                    ++c;
                    at.skip(1);
                }
            }
            ++pieces;
        }
        // the other CTA's last arrivals are in, and no MMA is left in flight
        if (ok && n > 0) warp_wait(sread(n - 1), ((n - 1) >> 1) & 1, abort_flag, 20);
        if (elect_one())
            asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(drain_s)
                         : "memory");
        __syncwarp();
        warp_wait(drain_s, 0, abort_flag, 21);
        __syncwarp();
    } else if (warp == PC_WARP_PV && cta == 0) {
        // ------------------------------------------------------------ O += P . tile for the pair
        constexpr uint32_t IDESC_PV = idesc_bf16(PC_ROWS, 256, 0, 1);
        const uint64_t p_desc = sdesc_sw128(sbase + PC_OFF_P, 16, 1024), v_desc = sdesc_sw128(vaddr(0), 1024, 4096);
        // 16-row parts v .. v + count - 1 of a tile, from slot `at` on
        const auto pv_mmas = [&](RingPlace<PC_VRING> at, int v, int count, bool add) {
#pragma unroll 1
            for (; count > 0; --count, ++v, ++at) {
                const uint64_t p = p_desc + uint64_t((v >> 2) * (8192 >> 4) + (v & 3) * 2);
                const uint64_t vd = v_desc + uint64_t(at.slot * (PC_SLOT >> 4));
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    mma2_ss(tmem + PC_TM_O + 128 * j, p, vd + 128 * j, IDESC_PV, add || v > 0 ? 1u : 0u);
                tc_commit_pair(vempty(at.slot));
            }
        };
        RingPlace<PC_VRING> at;
        uint32_t n = 0, pieces = 0;
        bool ok = true;
        while (ok && range.next(a.plan, w)) {
            const int m = __shfl_sync(0xffffffffu, w.n(), 0);
            if (m == 0) continue;
            const int32_t nv_all = clamp_rows(w.t.row_base + w.t.t0, max_rows);
            for (int i = 0; i < m && ok; ++i, ++n) {
                const int nvs = __shfl_sync(0xffffffffu, w.v_slots(i, max_rows), 0);
                if (int64_t(w.k0 + i + 1) * PC_TILE > nv_all) {
                    // an edge tile (see the softmax): its rows have landed
                    RingPlace<PC_VRING> x = at;
#pragma unroll 1
                    for (int v = 0; v < nvs && ok; ++v, ++x) ok = warp_wait(vfull(x.slot), x.par, abort_flag, 11);
                    if (!ok) break;
                    if (lane < 2) mbar_arrive_pair(map_to_cta(vready, lane));
                    __syncwarp();
                }
                if (i == 0 && !(ok = warp_wait(oread, (pieces & 1) ^ 1, abort_flag, 12))) break;
                if (!(ok = warp_wait(pfull(n), (n >> 1) & 1, abort_flag, 13))) break;
                bool looked = at.look(vfull(0), 0, lane);
                for (int v = 0; v < nvs;) {
                    const int got = min(at.count(vfull(0), looked, abort_flag, 14), nvs - v);
                    if (!(ok = got > 0)) break;
                    tc_fence_after();
                    if (got > 1 && elect_one()) pv_mmas(at, v, got - 1, i > 0);
                    __syncwarp();
                    v += got - 1;
                    at.skip(uint32_t(got - 1));
                    looked = at.look(vfull(0), 1, lane);
                    if (elect_one()) {
                        pv_mmas(at, v, 1, i > 0);
                        if (v + 1 == nvs) tc_commit_pair(vdone(n));
                    }
                    __syncwarp();
                    ++v;
                    at.skip(1);
                }
            }
            ++pieces;
        }
        if (ok && pieces > 0) warp_wait(oread, (pieces - 1) & 1, abort_flag, 22);
        if (elect_one())
            asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(drain_pv)
                         : "memory");
        __syncwarp();
        warp_wait(drain_pv, 0, abort_flag, 24);
        __syncwarp();
    } else if (warp < PC_SOFTMAX) {
        // ------------------------------------------------------------ softmax and epilogue
        // (half: which 64 of the tile's rows and 256 of o's columns.)  Once a
        // wait has given up (!ok) the loops run on without waiting or arriving
        // anywhere but at the pair's named barrier.
        const int lane4 = 32 * warp + lane, row = lane4 & 63, half = lane4 >> 6;
        const uint32_t lane_base = uint32_t(32 * warp) << 16;
        const int pair_bar = 1 + (warp & 1);   // warps w and w + 2 share their rows
        float *xm = reinterpret_cast<float *>(smem + PC_OFF_X);
        const int tok = 4 * int(cta) + (row >> 4);
        const uint32_t peer_sread = map_to_cta(sread(0), 0), peer_pfull = map_to_cta(pfull(0), 0);
        const uint32_t peer_oread = map_to_cta(oread, 0);
        const int sub_shift = min(a.page_shift, 7), subs = PC_TILE >> sub_shift;
        const uint32_t all_pages = (1u << subs) - 1u;
        uint32_t n = 0, x0 = 0, edges = 0, swaps = 0;   // x0: first use of PV's ring
        bool ok = true;
        // The value of the other thread of this row.  Two buffers in turn: who
        // writes one has seen the other past the exchange that used it last.
        const auto exchange = [&](float v) {
            float *x = xm + (swaps++ & 1) * 128;
            x[lane4] = v;
            named_bar_sync(pair_bar, 64);
            return x[lane4 ^ 64];
        };
        while (range.next(a.plan, w)) {
            const int tiles = w.n();
            const int32_t t = w.t.t0 + tok;
            const bool live = tok < w.t.live;
            const int32_t nv = live ? clamp_rows(w.t.row_base + t, max_rows) : 0;
            // rows that every live token of the tile (of both CTAs) attends
            const int32_t nv_all = clamp_rows(w.t.row_base + w.t.t0, max_rows);
            const int nvs_last = tiles ? w.v_slots(tiles - 1, max_rows) : 0;
            float m = NO_ROW, l = 0.f;
            int32_t row0 = w.k0 * PC_TILE;
            // lane c looks up the c-th of a tile's pages, a tile ahead
            const int32_t *table = a.block_table + size_t(w.t.b) * size_t(a.max_blocks);
            const auto page_of = [&](int32_t r) {
                const int32_t k = (r >> a.page_shift) + (a.page_shift < 7 ? lane : 0);
                return lane < subs && k < int32_t(a.max_blocks) ? __ldg(table + k) : -1;
            };
            int32_t page = tiles ? page_of(row0) : -1;
            for (int i = 0; i < tiles; ++i, ++n, row0 += PC_TILE) {
                const uint32_t pages = __ballot_sync(0xffffffffu, uint32_t(page) < uint32_t(a.n_pages));
                if (i + 1 < tiles) page = page_of(row0 + PC_TILE);
                ok = ok && warp_wait(sdone(n), (n >> 1) & 1, abort_flag, 15);
                tc_fence_after();
                float s[64];
                tmem_ld64(tmem + lane_base + PC_TM_S + 64 * (n & 1), s);
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive_pair(peer_sread + 8 * (n & 1));

                const bool edge = row0 + PC_TILE > nv_all;   // the same for both CTAs
                bool v_due = false;
                if (edge) {
                    // A row that is not attended by every token enters their
                    // PV product with weight 0, which a NaN or infinity in
                    // its latent would turn into NaN.  Such a row makes every
                    // logit against it non-finite: look those rows up and
                    // clear what is not finite in this CTA's columns of them
                    // (a token that does attend the row has the NaN in its
                    // weight already, unless its logit is minus infinity,
                    // which leaves the row out).
                    const int nvs = i + 1 == tiles ? nvs_last : PC_VS;
                    bool waited = false;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t odd = 0;
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (!(fabsf(s[32 * h + x]) <= 3.4e38f)) odd |= 1u << x;
                        odd = __reduce_or_sync(0xffffffffu, odd);
                        if (odd && !waited) {
                            ok = ok && warp_wait(vready, edges & 1, abort_flag, 16);
                            waited = true;
                        }
                        while (odd && ok) {
                            const int r = 64 * half + 32 * h + __ffs(int(odd)) - 1;
                            odd &= odd - 1;
                            if ((r >> 4) >= nvs) break;
                            uint4 *p = reinterpret_cast<uint4 *>(smem + (vaddr((x0 + (r >> 4)) % PC_VRING) - sbase) +
                                                                 ((r >> 3) & 1) * 4096 + (lane >> 3) * 1024 +
                                                                 (r & 7) * 128 + (lane & 7) * 16);
                            const uint4 v = *p;
                            bool bad = false;
                            for (uint32_t e : {v.x, v.y, v.z, v.w})
                                bad |= (e & 0x7f80u) == 0x7f80u || (e & 0x7f800000u) == 0x7f800000u;
                            if (__any_sync(0xffffffffu, bad)) *p = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    v_due = !waited;
                }
                if (edge || !live || pages != all_pages) {
                    const int32_t left = nv - row0 - 64 * half;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int32_t k = left - 32 * h;
                        uint32_t in = k <= 0 ? 0u : k >= 32 ? ~0u : (1u << k) - 1u;
#pragma unroll
                        for (int c = 0; c < 2; ++c)   // 16 rows lie in one page
                            if (!((pages >> ((64 * half + 32 * h + 16 * c) >> sub_shift)) & 1u)) in &= ~(0xffffu << (16 * c));
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (!((in >> x) & 1u)) s[32 * h + x] = -INFINITY;
                    }
                }
                float tm[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int x = 4; x < 64; x += 8)
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        tm[y] = x + 4 + y < 64 ? fmaxf(fmaxf(tm[y], s[x + y]), s[x + 4 + y]) : fmaxf(tm[y], s[x + y]);
                float tmax = fmaxf(fmaxf(tm[0], tm[1]), fmaxf(tm[2], tm[3]));
                tmax = fmaxf(tmax, exchange(tmax)) * a.sl2;
                float f = 1.f;
                if (i == 0) {
                    m = fmaxf(tmax, NO_ROW);
                } else if (tmax > m + 8.f) {
                    f = fast_exp2(m - tmax);
                    m = tmax;
                    l *= f;
                }
                const float shrink = shrink_of(m), mul = a.sl2 * shrink, off = m * -shrink;
                const uint64_t scale = pack2(mul, mul), shift = pack2(off, off);
                uint64_t sum[2] = {0, 0};
                uint32_t pk[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    float p0, p1;
                    unpack2(fma2(pack2(s[2 * x], s[2 * x + 1]), scale, shift), p0, p1);
                    p0 = fast_exp2(p0);
                    p1 = fast_exp2(p1);
                    sum[x & 1] = add2(sum[x & 1], pack2(p0, p1));
                    pk[x] = pack_bf16(p0, p1);
                }
                float sum0, sum1;
                unpack2(add2(sum[0], sum[1]), sum0, sum1);
                l += sum0 + sum1;
                // P(n - 1) has been used, and O holds PV(n - 1)
                if (n > 0) ok = ok && warp_wait(vdone(n - 1), ((n - 1) >> 1) & 1, abort_flag, 17);
                uint8_t *prow = smem + PC_OFF_P + half * 8192 + (row >> 3) * 1024 + (row & 7) * 128;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    *reinterpret_cast<uint4 *>(prow + ((e ^ (row & 7)) << 4)) =
                        make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
                fence_proxy_async();
                // every edge tile's arrival is taken, so that the next one's can be told apart
                if (v_due) ok = ok && warp_wait(vready, edges & 1, abort_flag, 16);
                if (edge) ++edges;
                if (__any_sync(0xffffffffu, f != 1.f)) {
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
                if (lane == 0 && ok) mbar_arrive_pair(peer_pfull + 8 * (n & 1));
                x0 += uint32_t(PC_VS);
            }
            x0 += uint32_t(nvs_last - (tiles ? PC_VS : 0));

            // ---- this thread's half row: columns 256 half .. + 255
            if (tiles) {
                l += exchange(l);
                ok = ok && warp_wait(vdone(n - 1), ((n - 1) >> 1) & 1, abort_flag, 23);
                tc_fence_after();
            }
            // Rows leave through this warp's quarter of the P buffer (free: PV is
            // done), 128 bytes of each at a time, so that a store instruction
            // writes four whole lines: straight from the registers, 32 bytes of 32
            // rows at once, they took 10000 cycles for a query tile.
            const float inv = l == 0.f ? 0.f : 1.f / l;
            if (w.slot >= 0 && half == 0)
                *reinterpret_cast<float2 *>(a.part_ml + (size_t(w.slot) * PC_ROWS + 64 * cta + row) * 2) =
                    make_float2(m, l);
            uint8_t *stage = smem + PC_OFF_P + warp * 4096;
            const int row_w = row & 32;                                          // the warp's first row
            const int rows_live = LCA_HEADS * (w.t.live - 4 * int(cta)) - row_w;   // of the warp's 32
            // 128 bytes of each of the warp's rows, `pitch` bytes apart from `dst` on
            const auto store_lines = [&](const uint32_t (&v)[32], void *dst, int pitch) {
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    *reinterpret_cast<uint4 *>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) =
                        make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                __syncwarp();
                uint4 x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = 4 * e + (lane >> 3);
                    x[e] = *reinterpret_cast<const uint4 *>(stage + i * 128 + (((lane & 7) ^ (i & 7)) << 4));
                }
                uint8_t *line = static_cast<uint8_t *>(dst) + (lane >> 3) * pitch + (lane & 7) * 16;
#pragma unroll
                for (int e = 0; e < 8; ++e, line += 4 * pitch)
                    if (4 * e + (lane >> 3) < rows_live) *reinterpret_cast<uint4 *>(line) = x[e];
            };
            const int chunks = w.slot >= 0 ? 8 : 4;   // 32 columns of fp32, or 64 of hi and of lo
#pragma unroll 1
            for (int c = 0; c < chunks && rows_live > 0; ++c) {
                float o[32];
                uint32_t x[32];
                const auto load = [&](int col) {
                    if (tiles) {
                        tmem_ld32(tmem + lane_base + PC_TM_O + col, o);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0.f;
                    }
                };
                if (w.slot >= 0) {
                    load(32 * c);
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(o[e]);
                    store_lines(x, a.part_o + (size_t(w.slot) * PC_ROWS + 64 * cta + row_w) * LCA_DC + 256 * half + 32 * c,
                                LCA_DC * 4);
                } else {
                    uint32_t lo[32];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        load(64 * c + 32 * h);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float o0 = o[2 * e] * inv, o1 = o[2 * e + 1] * inv;
                            x[16 * h + e] = pack_bf16(o0, o1);
                            lo[16 * h + e] = pack_bf16(o0 - bf_lo(x[16 * h + e]), o1 - bf_hi(x[16 * h + e]));
                        }
                    }
                    // (rows of a query tile follow one another, token by token, head by head)
                    uint16_t *dst = a.o_hl + (size_t(w.t.t0 + 4 * int(cta)) * LCA_HEADS + row_w) * (2 * LCA_DC) +
                                    256 * half + 64 * c;
                    store_lines(x, dst, 4 * LCA_DC);
                    store_lines(lo, dst + LCA_DC, 4 * LCA_DC);
                }
            }
            if (tiles) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive_pair(peer_oread);
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
// Query tiles cut by a cluster's border: o = sum_s 2^(m_s - M) O_s /
// sum_s 2^(m_s - M) l_s per query row, one warp each (lane: 16 columns),
// written as hi + lo.  blockIdx.y + 1 is the first border inside the query
// tile, which starts in cluster c0 = blockIdx.y and has pieces of all clusters
// to c1.
constexpr int MG_THREADS = 256;

__global__ void __launch_bounds__(MG_THREADS) paged_merge_kernel(const ChunkArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    const ChunkPlan &p = a.plan;
    const int lane = threadIdx.x & 31;
    const int r = int(blockIdx.x) * (MG_THREADS / 32) + int(threadIdx.x >> 5);   // query row
    const ChunkMerge mg = p.merge[blockIdx.y + 1];
    if (mg.c1 < 0 || r / LCA_HEADS >= mg.live) return;
    const auto slot = [&](int k) { return size_t(k == mg.c0 ? 2 * k + 1 : 2 * k) * PC_ROWS + r; };
    float M = NO_ROW, den = 0.f, acc[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
    // 32 pieces at a time, a lane each: maximum, weight, sum; then all lanes the values
    for (int k0 = mg.c0; k0 <= mg.c1; k0 += 32) {
        const int k = k0 + lane;
        float2 ml = make_float2(NO_ROW, 0.f);
        if (k <= mg.c1) ml = *reinterpret_cast<const float2 *>(a.part_ml + slot(k) * 2);
        float top = ml.x;
#pragma unroll
        for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        top = fmaxf(top, M);
        const float old = fast_exp2(M - top);
        M = top;
        // a piece in which nothing is attended has weight 0, whatever its O
        const float f = ml.y == 0.f ? 0.f : fast_exp2(ml.x - M);
        float sum = f * ml.y;
#pragma unroll
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        den = fmaf(den, old, sum);
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] *= old;
        const int n = min(32, mg.c1 - k0 + 1);
        // (four pieces' values asked for together; the build's 54 registers
        // hold about half of them at a time)
        for (int i0 = 0; i0 < n; i0 += 4) {
            float fi[4];
            float4 x[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                fi[i] = __shfl_sync(0xffffffffu, f, (i0 + i) & 31);
                if (i0 + i >= n) fi[i] = 0.f;
                const float4 *o = reinterpret_cast<const float4 *>(a.part_o + slot(k0 + i0 + i) * LCA_DC) + lane;
#pragma unroll
                for (int v = 0; v < 4; ++v)   // columns 128 v + 4 lane ..
                    x[i][v] = fi[i] == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : o[32 * v];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    acc[4 * v] = fmaf(fi[i], x[i][v].x, acc[4 * v]);
                    acc[4 * v + 1] = fmaf(fi[i], x[i][v].y, acc[4 * v + 1]);
                    acc[4 * v + 2] = fmaf(fi[i], x[i][v].z, acc[4 * v + 2]);
                    acc[4 * v + 3] = fmaf(fi[i], x[i][v].w, acc[4 * v + 3]);
                }
        }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    uint16_t *hl = a.o_hl + (size_t(mg.t0 + r / LCA_HEADS) * LCA_HEADS + r % LCA_HEADS) * (2 * LCA_DC) + 4 * lane;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float o0 = acc[4 * v + 2 * e] * inv, o1 = acc[4 * v + 2 * e + 1] * inv;
            hi[e] = pack_bf16(o0, o1);
            lo[e] = pack_bf16(o0 - bf_lo(hi[e]), o1 - bf_hi(hi[e]));
        }
        *reinterpret_cast<uint2 *>(hl + 128 * v) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2 *>(hl + LCA_DC + 128 * v) = make_uint2(lo[0], lo[1]);
    }
}

}  // namespace lca
