// paged_wuv.cuh -- the value up-projection behind the chunk kernel:
// out[t, h] = W_UV[h]^T (o_hi + o_lo)[t, h], bf16 in and out, fp32 sums.
//
// o comes as two bf16 values per element, [T][16][hi 512 | lo 512], and enters
// the product to 2^-16: the only roundings to bf16 between the logits and the
// result are the weights' and the result's own.  One CTA computes 128 tokens x
// 128 columns of one head; a stage is 64 of the 512 latent columns of hi, of lo
// and of W_UV[h], which both share.  Two stages of 48 KB, so that two CTAs fit
// an SM and one's epilogue runs under the other's loads.
//
// What bounds it: the bytes of o, 32 KB a token (4 B per element as fp32 would
// have, hi + lo being as much) from L2 or memory.
#pragma once
#include "paged_chunk.cuh"

namespace lca {

constexpr int PW_STAGES = 2;
constexpr int PW_A = 128 * 128;            // 16 KB: [128 tokens x 64] bf16
constexpr int PW_B = 2 * 64 * 128;         // 16 KB: 2 x [64 x 64 columns]
constexpr int PW_STAGE = 2 * PW_A + PW_B;
constexpr int PW_OFF_BAR = PW_STAGES * PW_STAGE;
constexpr int PW_SMEM_ALLOC = PW_OFF_BAR + 128 + 1024;
static_assert(2 * (PW_SMEM_ALLOC + 1024) <= 228 * 1024, "two CTAs per SM");
constexpr uint32_t PW_TM_COLS = 128;

__global__ void __launch_bounds__(128, 2)
    paged_wuv_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                     uint16_t *__restrict__ out, int64_t T, const int32_t *__restrict__ q_start, int B)
{
    extern __shared__ uint8_t pw_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(pw_smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mt = blockIdx.x, h = blockIdx.y;
    constexpr int KC = LCA_DC / 64;

    auto full = [&](int s) -> uint32_t { return sbase + PW_OFF_BAR + 8 * s; };
    auto empty = [&](int s) -> uint32_t { return sbase + PW_OFF_BAR + 8 * (PW_STAGES + s); };
    const uint32_t accf = sbase + PW_OFF_BAR + 8 * (2 * PW_STAGES), drain = accf + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + PW_OFF_BAR + 96);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + PW_OFF_BAR + 100);

    if (threadIdx.x == 0) {
        for (int s = 0; s < PW_STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(accf, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), PW_TM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&map_a);
        prefetch_tensormap(&map_b);
        const uint64_t pa = policy_evict_first(), pb = policy_evict_last();
        const auto load_w = [&](int kc) {
            const int s = kc % PW_STAGES;
            mbar_expect_tx(full(s), PW_STAGE);
            tma_load_3d(sbase + s * PW_STAGE + 2 * PW_A, &map_b, full(s), 0, 64 * kc, h, pb);
            tma_load_3d(sbase + s * PW_STAGE + 2 * PW_A + 8192, &map_b, full(s), 64, 64 * kc, h, pb);
        };
        // W_UV's first stages before the kernel in front is done: it was
        // written by nothing later than the kernels that one has waited for
        for (int kc = 0; kc < PW_STAGES; ++kc) load_w(kc);
        griddep_wait();   // o comes from the kernel before
        griddep_launch_dependents();
        int last[PW_STAGES];
        for (int kc = 0; kc < KC; ++kc) {
            const int s = kc % PW_STAGES;
            if (kc >= PW_STAGES) {
                if (!mbar_wait(empty(s), ((kc / PW_STAGES) & 1) ^ 1, abort_flag, K_GEMM, 9)) break;
                load_w(kc);
            }
            tma_load_3d(sbase + s * PW_STAGE, &map_a, full(s), 64 * kc, h, mt * 128, pa);
            tma_load_3d(sbase + s * PW_STAGE + PW_A, &map_a, full(s), LCA_DC + 64 * kc, h, mt * 128, pa);
            last[s] = kc;
        }
        for (int s = 0; s < PW_STAGES; ++s) mbar_wait(full(s), (last[s] / PW_STAGES) & 1, nullptr, K_GEMM, 10);
    } else {
        griddep_wait();
        griddep_launch_dependents();
        if (warp == 1 && lane == 0) {
            constexpr uint32_t IDESC = idesc_bf16(128, 128, 0, 1);
            bool ok = true;
            for (int kc = 0; kc < KC && ok; ++kc) {
                const int s = kc % PW_STAGES;
                if (!(ok = mbar_wait(full(s), (kc / PW_STAGES) & 1, abort_flag, K_GEMM, 11))) break;
                tc_fence_after();
                const uint32_t st = sbase + s * PW_STAGE;
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_ss(tmem, sdesc_sw128(st + part * PW_A + ks * 32, 16, 1024),
                               sdesc_sw128(st + 2 * PW_A + ks * 2048, 8192, 1024), IDESC, (kc | part | ks) ? 1u : 0u);
                tc_commit(empty(s));
            }
            if (ok) tc_commit(accf);
            tc_commit(drain);
            mbar_wait(drain, 0, nullptr, K_GEMM, 12);
        }
    }
    __syncwarp();

    // lane = token of the tile, 128 columns each; rows of no sequence are left as they were
    bool ok = mbar_wait(accf, 0, abort_flag, K_GEMM, 13);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
        tc_fence_after();
        const int64_t row = int64_t(mt) * 128 + 32 * warp + lane;
        const bool live = row >= q_start[0] && row < min64(T, q_start[B]);
        const uint32_t ta = tmem + (uint32_t(32 * warp) << 16);
#pragma unroll 1
        for (int cc = 0; cc < 4; ++cc) {
            float v[32];
            tmem_ld32(ta + 32 * cc, v);
            if (!live) continue;
            uint16_t *dst = out + (size_t(row) * LCA_HEADS + h) * LCA_DV + 32 * cc;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                reinterpret_cast<uint4 *>(dst)[e] =
                    make_uint4(pack_bf16(v[8 * e], v[8 * e + 1]), pack_bf16(v[8 * e + 2], v[8 * e + 3]),
                               pack_bf16(v[8 * e + 4], v[8 * e + 5]), pack_bf16(v[8 * e + 6], v[8 * e + 7]));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, PW_TM_COLS);
}

}  // namespace lca
