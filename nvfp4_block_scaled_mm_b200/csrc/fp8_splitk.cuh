// E4M3 x E4M3 product with fp32 scales per block of 128 for few rows, or few tiles (sm_100a).
//
// The operation of fp8_gemm.cuh with the operands swapped: the weight rows take the MMA's 128 lanes
// and the tokens its MT columns, so that few tokens leave no tensor-core rows empty, and K is split
// over a cluster of S CTAs, so that few weight rows still stream from every SM:
//   * CTA r of a cluster takes the K blocks [kb r / S, kb (r + 1) / S) of one 128 x MT tile: a TMA
//     ring of 128 x 128 weight tiles and MT x 128 token tiles, one MMA thread (kind::f8f6f4, M = 128,
//     N = MT, four K = 32 steps per block), each block's product into the next of NB accumulators;
//   * four warps read each product back and add it to fp32 sums, acc[m] += (sa[m, kb] sb[kb]) * P[m];
//     a lane is a weight row, so the CTA's products of scales, one per token and block, are staged in
//     shared memory eight blocks at a time and read as broadcasts;
//   * the S partial sums meet in distributed shared memory: CTA r receives every CTA's share of the
//     token columns [MT r / S, MT (r + 1) / S), adds them in rank order and rounds once, so the result
//     does not depend on the schedule.
// At a decode step the kernel is bound by streaming the weights from HBM.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "fp8_gemm.cuh"
#include "ptx.cuh"

namespace nvfp4lora {

constexpr int kSplitThreads = 192;       // warp 0: producer, 1: MMA issuer, 2..5: promotion
constexpr int kSplitMaxS = 8;
constexpr int kSplitScaleChunk = 8;      // K blocks whose scale products are staged at a time

struct Fp8SplitArgs {
    const float* a_scale;    // element (m, kb) at m * stride_am + kb * stride_ak
    const float* b_scale;    // [ceil(N / 128), kblocks]
    const uint16_t* bias;    // bf16 [N] or null
    void* out;               // [M, N]
    int64_t stride_am, stride_ak;
    int M, N, kblocks, splits;
};

template <int MT>
struct Fp8SplitPlan {
    static constexpr int W_BYTES = 128 * 128;
    static constexpr int X_BYTES = MT * 128;
    // MT <= 64: two CTAs per SM (shared memory, registers and TMEM allow both)
    static constexpr int STAGES = MT == 16 ? 6 : MT == 32 ? 5 : MT == 64 ? 4 : 6;
    static constexpr int NB = MT <= 32 ? 8 : MT == 64 ? 4 : 2;        // accumulators
    static constexpr int TMEM_COLS = NB * MT;                         // 128 or 256: a power of two
    static constexpr int W_OFF = 0;
    static constexpr int X_OFF = W_OFF + STAGES * W_BYTES;
    static constexpr int SC_OFF = X_OFF + STAGES * X_BYTES;           // [2][chunk][MT] scale products
    static constexpr int BAR_OFF = SC_OFF + 2 * kSplitScaleChunk * MT * 4;
    static constexpr int NUM_BARS = 2 * STAGES + 2 * NB + 1;          // full, empty, acc_full, acc_empty, drain
    static constexpr int MISC_OFF = BAR_OFF + NUM_BARS * 8;
    static constexpr int TOTAL = MISC_OFF + 16;
    static constexpr int DYN_BYTES = TOTAL + 1024;
    // the partial sums of the exchange take the ring's place: S x ceil(MT / S) x 128 floats
    static_assert((MT + kSplitMaxS) * 128 * 4 <= STAGES * (W_BYTES + X_BYTES), "partials exceed the ring");
    static_assert(X_BYTES % 1024 == 0, "token tiles must stay 1024-byte aligned");
    static_assert(DYN_BYTES <= (MT <= 64 ? 113 * 1024 : 227 * 1024), "split-K shared-memory plan too large");
};

__device__ __forceinline__ void st_cluster_f32(uint32_t caddr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(caddr), "f"(v) : "memory");
}

constexpr uint32_t kSplitScaleBarrier = 1;       // named barrier: the four promotion warps

template <int MT, OutType OT>
__global__ void __launch_bounds__(kSplitThreads, MT <= 64 ? 2 : 1)
fp8_splitk_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                  const Fp8SplitArgs args) {
    using L = Fp8SplitPlan<MT>;
    constexpr uint32_t IDESC = idesc_e4m3_m(128, MT);
    constexpr uint32_t kAll = 0xffffffffu;
    constexpr int CH = kSplitScaleChunk;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
    uint64_t* empty = full + L::STAGES;
    uint64_t* acc_full = empty + L::STAGES;
    uint64_t* acc_empty = acc_full + L::NB;
    uint64_t* drain = acc_empty + L::NB;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC_OFF + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int n_blk = blockIdx.x;
    const int m0 = blockIdx.z * MT;
    const int S = args.splits;
    const bool clustered = S > 1;
    const uint32_t rank = clustered ? cluster_rank() : 0u;
    const int k0 = (int)((int64_t)args.kblocks * rank / S);
    const int k1 = (int)((int64_t)args.kblocks * (rank + 1) / S);

    if (threadIdx.x == 0) {
        prefetch_tensor_map(&tm_b);
        prefetch_tensor_map(&tm_a);
        for (int s = 0; s < L::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < L::NB; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, L::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // the next grid's CTAs may take this SM's remaining TMEM only after this CTA has its own
    grid_launch_dependents();

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------- TMA producer -------------------------------
            // A prefetch changes no data and L2 is where device memory is kept coherent, so the weights
            // of the ring's first fill may be warmed before the dependency wait.
            for (int kb = k0; kb < min(k1, k0 + L::STAGES); ++kb) tma_prefetch_l2_2d(&tm_b, kb * 128, n_blk * 128);
            grid_dependency_wait();
            int stage = 0;
            uint32_t phase = 0, filled = 0, filled_parity = 0;
            bool ok = true;
            for (int kb = k0; kb < k1; ++kb) {
                if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) { ok = false; break; }
                mbar_arrive_expect_tx(&full[stage], L::W_BYTES + L::X_BYTES);
                tma_load_2d(smem + L::W_OFF + stage * L::W_BYTES, &tm_b, &full[stage], kb * 128, n_blk * 128);
                tma_load_2d(smem + L::X_OFF + stage * L::X_BYTES, &tm_a, &full[stage], kb * 128, m0);
                filled |= 1u << stage;
                filled_parity = (filled_parity & ~(1u << stage)) | (phase << stage);
                if (++stage == L::STAGES) { stage = 0; phase ^= 1; }
            }
            if (!ok || *abort_flag) {
                // Let the copies already issued land before the CTA can exit.
                for (int s = 0; s < L::STAGES; ++s)
                    if ((filled >> s) & 1u) mbar_wait(&full[s], (filled_parity >> s) & 1u, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            // ------------------------------- MMA issuer ---------------------------------
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int i = 0; i < k1 - k0; ++i) {
                const int buf = i % L::NB;
                if (!mbar_wait(&acc_empty[buf], ((i / L::NB) & 1) ^ 1, abort_flag)) { ok = false; break; }
                if (!mbar_wait(&full[stage], phase, abort_flag)) { ok = false; break; }
                tc_fence_after();
                const uint32_t w_addr = smem_u32(smem + L::W_OFF + stage * L::W_BYTES);
                const uint32_t x_addr = smem_u32(smem + L::X_OFF + stage * L::X_BYTES);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    tc_mma_fp8(tmem + buf * MT, sdesc_sw128(w_addr + j * 32), sdesc_sw128(x_addr + j * 32), IDESC,
                               j > 0 ? 1u : 0u);
                tc_commit(&empty[stage]);
                tc_commit(&acc_full[buf]);
                if (++stage == L::STAGES) { stage = 0; phase ^= 1; }
            }
            if (!ok || *abort_flag) {
                tc_commit(drain);
                mbar_wait(drain, 0, nullptr);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------- promotion -----------------------------------
        const int q = warp & 3;
        const int et = threadIdx.x - 64;              // 0..127
        const int nl = q * 32 + lane;                 // weight row within the tile = TMEM lane
        const int n = n_blk * 128 + nl;               // output column
        const uint32_t lane_off = (uint32_t)(q * 32) << 16;
        float* sc = reinterpret_cast<float*>(smem + L::SC_OFF);
        grid_dependency_wait();
        const float* sb = args.b_scale + (int64_t)n_blk * args.kblocks;
        const float bias_v = (args.bias != nullptr && n < args.N) ? __uint_as_float((uint32_t)__ldg(args.bias + n) << 16)
                                                                  : 0.0f;
        // the scale products of a chunk of K blocks: MT x CH values over 128 threads
        constexpr int PER = MT * CH / 128;
        float pre[PER];
        auto fetch = [&](int kc) {
#pragma unroll
            for (int v = 0; v < PER; ++v) {
                const int idx = v * 128 + et, m = m0 + idx % MT, kb = kc + idx / MT;
                pre[v] = (m < args.M && kb < k1)
                             ? __ldg(args.a_scale + m * args.stride_am + kb * args.stride_ak) * __ldg(sb + kb) : 0.0f;
            }
        };
        float acc[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m] = 0.0f;
        bool ok = true;
        fetch(k0);
        for (int kc = k0, ci = 0; kc < k1; kc += CH, ++ci) {
            // this buffer was last read two chunks ago, before every thread's previous barrier
            float* cur = sc + (ci & 1) * CH * MT;
#pragma unroll
            for (int v = 0; v < PER; ++v) cur[v * 128 + et] = pre[v];
            named_barrier_sync(kSplitScaleBarrier, 128);
            fetch(kc + CH);
            const int ke = min(CH, k1 - kc);
            for (int j = 0; j < ke; ++j) {
                const int i = kc - k0 + j, buf = i % L::NB;
                if (ok) ok = __all_sync(kAll, mbar_wait(&acc_full[buf], (i / L::NB) & 1, abort_flag));
                if (!ok) break;
                tc_fence_after();
                const float4* s4 = reinterpret_cast<const float4*>(cur + j * MT);
                constexpr int W = MT < 32 ? 16 : 32;   // columns per read
#pragma unroll
                for (int c = 0; c < MT; c += W) {
                    uint32_t p[W];
                    if constexpr (W == 32) tmem_load_32(tmem + lane_off + buf * MT + c, p);
                    else tmem_load_16(tmem + lane_off + buf * MT + c, p);
                    tmem_load_wait();
                    if (c + W == MT) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&acc_empty[buf]);
                    }
#pragma unroll
                    for (int m = 0; m < W; m += 4) {
                        const float4 s = s4[(c + m) / 4];
                        acc[c + m] = fmaf(s.x, __uint_as_float(p[m]), acc[c + m]);
                        acc[c + m + 1] = fmaf(s.y, __uint_as_float(p[m + 1]), acc[c + m + 1]);
                        acc[c + m + 2] = fmaf(s.z, __uint_as_float(p[m + 2]), acc[c + m + 2]);
                        acc[c + m + 3] = fmaf(s.w, __uint_as_float(p[m + 3]), acc[c + m + 3]);
                    }
                }
            }
        }
        if (!clustered) {
            if (ok && n < args.N) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    if (m0 + m < args.M)
                        store_out_one<OT>(args.out, (int64_t)(m0 + m) * args.N + n,
                                          args.bias != nullptr ? __fadd_rn(acc[m], bias_v) : acc[m]);
            }
        } else {
            // every CTA's MMAs have read their ring: its memory takes the partial sums now
            float* part = reinterpret_cast<float*>(smem);
            const int cw = (MT + S - 1) / S;              // columns per owner, at most
            cluster_arrive();
            cluster_wait();
            int r = 0, c0 = 0, c1 = MT / S;               // owner r has the columns [MT r / S, MT (r + 1) / S)
            uint32_t dst = map_to_rank(smem_u32(part + (size_t)rank * cw * 128 + nl), 0);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                while (m >= c1) {
                    ++r;
                    c0 = c1;
                    c1 = MT * (r + 1) / S;
                    dst = map_to_rank(smem_u32(part + (size_t)rank * cw * 128 + nl), (uint32_t)r);
                }
                st_cluster_f32(dst + (uint32_t)(m - c0) * 512u, acc[m]);
            }
            cluster_arrive();
            cluster_wait();
            const int b0 = MT * (int)rank / S, b1 = MT * ((int)rank + 1) / S;
            if (ok && n < args.N) {
                for (int m = b0; m < b1 && m0 + m < args.M; ++m) {
                    const float* src = part + (size_t)(m - b0) * 128 + nl;
                    float v = src[0];
                    for (int p = 1; p < S; ++p) v = __fadd_rn(v, src[(size_t)p * cw * 128]);
                    if (args.bias != nullptr) v = __fadd_rn(v, bias_v);
                    store_out_one<OT>(args.out, (int64_t)(m0 + m) * args.N + n, v);
                }
            }
        }
    }
    if (clustered && warp < 2) {
        // one arrive / wait pair per thread for each of the two meetings above
        cluster_arrive();
        cluster_wait();
        cluster_arrive();
        cluster_wait();
    }
    // every read of the accumulators lies before this point
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L::TMEM_COLS);
    }
}

}  // namespace nvfp4lora
