// E4M3 x E4M3 product with fp32 scales per block of 128 for few rows, or few tiles (sm_100a).
//
// The operation of fp8_gemm.cuh with the operands swapped: the weight rows take the MMA's 128 lanes
// and the tokens its MT columns, so that few tokens leave no tensor-core rows empty, and K is split
// over a cluster of S CTAs, so that few weight rows still stream from every SM:
//   * CTA r of a cluster takes the K blocks [kb r / S, kb (r + 1) / S) of one 128 x MT tile: a TMA
//     ring of 128 x 128 weight tiles and MT x 128 token tiles, two MMA-issuing warps that take the blocks in
//     turn (kind::f8f6f4, M = 128, N = MT, four K = 32 steps per block), each block's product into the next of
//     NB accumulators;
//   * promotion warps read each product back and add it to fp32 sums, acc[m] += (sa[m, kb] sb[kb]) * P[m];
//     a lane is a weight row, so the CTA's products of scales, one per token and block, are staged in
//     shared memory eight blocks at a time and read as broadcasts;
//   * the S partial sums meet in distributed shared memory: CTA r reads every CTA's sums of the token
//     columns [MT r / S, MT (r + 1) / S), adds them in rank order and rounds once, so the result does
//     not depend on the schedule.
// 80 registers at two CTAs per SM; with MT = 64 a thread spills 4 bytes.
// Bound by streaming the weights from HBM where there are many: 16 x 28672 x 8192 runs 40 us (5.9 TB/s of the
// measured 6.46).  At 16 x 4096 x 4096 (17 MB, 6.9 us) the stream itself takes 2.7 us at that rate; the rest is the
// first load's latency (0.9 us), the meeting of the partial sums (1.4 us) and the start and end of the grid.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "fp8_gemm.cuh"
#include "ptx.cuh"

namespace nvfp4lora {

constexpr int kSplitMaxS = 8;
constexpr int kSplitScaleChunk = 8;      // K blocks whose scale products are staged at a time
constexpr int kSplitIssuers = 2;         // MMA-issuing warps

struct Fp8SplitArgs {
    const float* a_scale;    // element (m, kb) at m * stride_am + kb * stride_ak
    const float* b_scale;    // [ceil(N / 128), kblocks]
    const uint16_t* bias;    // bf16 [N] or null
    void* out;               // [M, N]
    int64_t stride_am, stride_ak;
    int M, N, kblocks, splits;
    int vec_out;             // rows of out aligned to four elements
};

template <int MT>
struct Fp8SplitPlan {
    static constexpr int W_BYTES = 128 * 128;
    static constexpr int X_BYTES = MT * 128;
    // MT <= 64: two CTAs per SM (shared memory, registers and TMEM allow both)
    static constexpr int STAGES = MT == 16 ? 6 : MT == 32 ? 4 : MT == 64 ? 4 : 6;
    // promotion warps: one per TMEM lane quarter, two from 64 token columns on
    static constexpr int EW = MT >= 64 ? 8 : 4;
    static constexpr int THREADS = 96 + 32 * EW;                      // warp 0: producer, 1 and 2: MMA issuers
    static constexpr int COLS = MT * 4 / EW;                          // token columns per promotion thread
    static constexpr int NB = MT <= 32 ? 8 : MT == 64 ? 4 : 2;        // accumulators
    static constexpr int TMEM_COLS = NB * MT;                         // 128 or 256: a power of two
    static constexpr int W_OFF = 0;
    static constexpr int X_OFF = W_OFF + STAGES * W_BYTES;
    static constexpr int SC_OFF = X_OFF + STAGES * X_BYTES;           // [2][chunk][MT] scale products
    static constexpr int BAR_OFF = SC_OFF + 2 * kSplitScaleChunk * MT * 4;
    static constexpr int NUM_BARS = 2 * STAGES + 2 * NB + kSplitIssuers;   // full, empty, acc_full, acc_empty, drain
    static constexpr int MISC_OFF = BAR_OFF + NUM_BARS * 8;
    static constexpr int TOTAL = MISC_OFF + 16;
    static constexpr int DYN_BYTES = TOTAL + 1024;
    // the finished sums take the ring's place: [MT][128] floats
    static_assert(MT * 128 * 4 <= STAGES * (W_BYTES + X_BYTES), "partials exceed the ring");
    // a barrier's phases are all waited for by one issuer: a second one could be a whole phase ahead, where
    // the parity it waits for is that of the phase before
    static_assert(STAGES % kSplitIssuers == 0 && NB % kSplitIssuers == 0, "issuers must divide stages and accumulators");
    static_assert(X_BYTES % 1024 == 0, "token tiles must stay 1024-byte aligned");
    static_assert(DYN_BYTES <= (MT <= 64 ? 113 * 1024 : 227 * 1024), "split-K shared-memory plan too large");
};

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t caddr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(caddr) : "memory");
    return v;
}

// {a.x, a.y} + {s.x, s.y} * {p.x, p.y}, each rounded to nearest even (one packed fma)
__device__ __forceinline__ void fma2_pair(float& ax, float& ay, uint32_t px, uint32_t py, float sx, float sy) {
    uint64_t d;
    asm("{\n\t.reg .b64 pa, pp, ps;\n\t"
        "mov.b64 pa, {%1, %2};\n\t"
        "mov.b64 pp, {%3, %4};\n\t"
        "mov.b64 ps, {%5, %6};\n\t"
        "fma.rn.f32x2 %0, pp, ps, pa;\n\t}"
        : "=l"(d) : "f"(ax), "f"(ay), "r"(px), "r"(py), "f"(sx), "f"(sy));
    ax = __uint_as_float((uint32_t)d);
    ay = __uint_as_float((uint32_t)(d >> 32));
}

constexpr uint32_t kSplitScaleBarrier = 1;       // named barrier: the promotion warps

template <int MT, OutType OT>
__global__ void __launch_bounds__(Fp8SplitPlan<MT>::THREADS, MT <= 64 ? 2 : 1)
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
    volatile uint32_t* issued = reinterpret_cast<volatile uint32_t*>(smem + L::MISC_OFF + 8);   // K blocks copied

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
            mbar_init(&acc_empty[b], L::EW);
        }
        for (int k = 0; k < kSplitIssuers; ++k) mbar_init(&drain[k], 1);
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
        // ------------------------------- TMA producer -------------------------------
        // The ring's first fill is issued by a lane per stage (one lane alone takes about 340 cycles per
        // stage); lane 0 refills the stages as they are handed back.  A prefetch changes no data and L2 is
        // where device memory is kept coherent, so the weights of the first fill are warmed before the
        // dependency wait.
        const int mine = k0 + lane;
        const bool first = lane < L::STAGES && mine < k1;
        if (first) tma_prefetch_l2_2d(&tm_b, mine * 128, n_blk * 128);
        grid_dependency_wait();
        if (first) {
            mbar_arrive_expect_tx(&full[lane], L::W_BYTES + L::X_BYTES);
            tma_load_2d(smem + L::W_OFF + lane * L::W_BYTES, &tm_b, &full[lane], mine * 128, n_blk * 128);
            tma_load_2d(smem + L::X_OFF + lane * L::X_BYTES, &tm_a, &full[lane], mine * 128, m0);
        }
        __syncwarp();
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int kb = k0 + L::STAGES;
            for (; kb < k1; ++kb) {
                if (!mbar_wait_short(&empty[stage], phase, abort_flag)) break;
                mbar_arrive_expect_tx(&full[stage], L::W_BYTES + L::X_BYTES);
                tma_load_2d(smem + L::W_OFF + stage * L::W_BYTES, &tm_b, &full[stage], kb * 128, n_blk * 128);
                tma_load_2d(smem + L::X_OFF + stage * L::X_BYTES, &tm_a, &full[stage], kb * 128, m0);
                if (++stage == L::STAGES) { stage = 0; phase ^= 1; }
            }
            *issued = (uint32_t)(min(kb, k1) - k0);
        }
        __syncwarp();
    } else if (warp <= kSplitIssuers) {
        // ------------------------------- MMA issuers ---------------------------------
        // The blocks in turn: one warp's waits, vote and issue take about 700 cycles per block, more than
        // the block's MMAs or its share of the weight stream.
        bool ok = true;
        for (int i = warp - 1; i < k1 - k0; i += kSplitIssuers) {
            const int buf = i % L::NB, stage = i % L::STAGES;
            ok = mbar_wait_short(&full[stage], (i / L::STAGES) & 1, abort_flag) &&
                 (i < L::NB || mbar_wait_short(&acc_empty[buf], ((i / L::NB) & 1) ^ 1, abort_flag));
            if (!__all_sync(kAll, ok)) { ok = false; break; }
            tc_fence_after();
            const uint32_t w_addr = smem_u32(smem + L::W_OFF + stage * L::W_BYTES);
            const uint32_t x_addr = smem_u32(smem + L::X_OFF + stage * L::X_BYTES);
            if (elect_one()) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    tc_mma_fp8(tmem + buf * MT, sdesc_sw128(w_addr + j * 32), sdesc_sw128(x_addr + j * 32), IDESC,
                               j > 0 ? 1u : 0u);
                tc_commit(&acc_full[buf]);
                if (i + L::STAGES < k1 - k0) tc_commit(&empty[stage]);
            }
            __syncwarp();
        }
        if (!ok || *abort_flag) {
            // Wait for the MMAs already issued before TMEM is released.
            if (elect_one()) {
                tc_commit(&drain[warp - 1]);
                mbar_wait(&drain[warp - 1], 0, nullptr);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------- promotion -----------------------------------
        constexpr int ET = 32 * L::EW;
        const int q = warp & 3;
        const int et = threadIdx.x - 96;              // 0..ET - 1
        const int cb = (warp - 3) / 4 * L::COLS;      // this warp's first token column
        const int nl = q * 32 + lane;                 // weight row within the tile = TMEM lane
        const uint32_t lane_off = (uint32_t)(q * 32) << 16;
        float* sc = reinterpret_cast<float*>(smem + L::SC_OFF);
        grid_dependency_wait();
        const float* sb = args.b_scale + (int64_t)n_blk * args.kblocks;
        // the scales of a chunk of K blocks: MT x CH products over ET threads, loaded a chunk ahead and
        // multiplied when they are staged (a multiply at the load would stall the warp on it)
        constexpr int PER = MT * CH / ET;
        float pre_a[PER], pre_b[PER];
        auto fetch = [&](int kc) {
#pragma unroll
            for (int v = 0; v < PER; ++v) {
                const int idx = v * ET + et, m = m0 + idx % MT, kb = kc + idx / MT;
                const bool in = m < args.M && kb < k1;
                pre_a[v] = in ? args.a_scale[m * args.stride_am + kb * args.stride_ak] : 0.0f;
                pre_b[v] = in ? sb[kb] : 0.0f;
            }
        };
        float acc[L::COLS];
#pragma unroll
        for (int m = 0; m < L::COLS; ++m) acc[m] = 0.0f;
        bool ok = true;
        fetch(k0);
        for (int kc = k0, ci = 0; kc < k1; kc += CH, ++ci) {
            // this buffer was last read two chunks ago, before every thread's previous barrier
            float* cur = sc + (ci & 1) * CH * MT;
#pragma unroll
            for (int v = 0; v < PER; ++v) cur[v * ET + et] = pre_a[v] * pre_b[v];
            named_barrier_sync(kSplitScaleBarrier, ET);
            if (kc + CH < k1) fetch(kc + CH);
            const int ke = min(CH, k1 - kc);
            for (int j = 0; j < ke; ++j) {
                const int i = kc - k0 + j, buf = i % L::NB;
                if (ok) ok = __all_sync(kAll, mbar_wait_short(&acc_full[buf], (i / L::NB) & 1, abort_flag));
                if (!ok) break;
                tc_fence_after();
                const float4* s4 = reinterpret_cast<const float4*>(cur + j * MT + cb);
                constexpr int W = 16;                  // columns per read
#pragma unroll
                for (int c = 0; c < L::COLS; c += W) {
                    uint32_t p[W];
                    tmem_load_16(tmem + lane_off + buf * MT + cb + c, p);
                    tmem_load_wait();
                    if (c + W == L::COLS) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&acc_empty[buf]);
                    }
#pragma unroll
                    for (int m = 0; m < W; m += 4) {
                        const float4 s = s4[(c + m) / 4];
                        fma2_pair(acc[c + m], acc[c + m + 1], p[m], p[m + 1], s.x, s.y);
                        fma2_pair(acc[c + m + 2], acc[c + m + 3], p[m + 2], p[m + 3], s.z, s.w);
                    }
                }
            }
        }
        // The sums go through shared memory ([MT][128], in the place of the ring: the last acc_full says
        // that every MMA has read it), so that the code from here on is short loops: unrolled over the
        // registers it was fetched cold by every CTA, and that took longer than the product.
        float* part = reinterpret_cast<float*>(smem);
        if (ok) {
#pragma unroll
            for (int m = 0; m < L::COLS; ++m) part[(cb + m) * 128 + nl] = acc[m];
        }
        if (clustered) {
            cluster_arrive();
            cluster_wait();
        } else {
            named_barrier_sync(kSplitScaleBarrier, ET);
        }
        // this CTA's token columns, four weight rows per thread at a time
        const int b0 = MT * (int)rank / S, b1 = min(MT * ((int)rank + 1) / S, args.M - m0);
        const int n0 = n_blk * 128 + lane * 4;
        const bool vec = args.vec_out && n0 + 4 <= args.N;
        float4 bias = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (args.bias != nullptr) {
            float* bv = reinterpret_cast<float*>(&bias);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n0 + e < args.N) bv[e] = __uint_as_float((uint32_t)args.bias[n0 + e] << 16);
        }
        for (int m = b0 + et / 32; m < b1; m += L::EW) {
            float4 v;
            if (clustered) {
                const uint32_t src = smem_u32(part + m * 128 + lane * 4);
                // all reads are on their way before the first addition; rank order whatever S is
                float4 w[kSplitMaxS];
#pragma unroll
                for (int p = 0; p < kSplitMaxS; ++p)
                    if (p < S) w[p] = ld_cluster_v4(map_to_rank(src, (uint32_t)p));
                v = w[0];
#pragma unroll
                for (int p = 1; p < kSplitMaxS; ++p)
                    if (p < S)
                        v = make_float4(__fadd_rn(v.x, w[p].x), __fadd_rn(v.y, w[p].y), __fadd_rn(v.z, w[p].z),
                                        __fadd_rn(v.w, w[p].w));
            } else {
                v = reinterpret_cast<const float4*>(part + m * 128)[lane];
            }
            if (args.bias != nullptr)
                v = make_float4(__fadd_rn(v.x, bias.x), __fadd_rn(v.y, bias.y), __fadd_rn(v.z, bias.z), __fadd_rn(v.w, bias.w));
            if (!ok) continue;
            const int64_t at = (int64_t)(m0 + m) * args.N + n0;
            if (vec) {
                if constexpr (OT == OutType::FP32) *reinterpret_cast<float4*>(static_cast<float*>(args.out) + at) = v;
                else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(args.out) + at) =
                         make_uint2(pack_out2<OT>(v.x, v.y), pack_out2<OT>(v.z, v.w));
            } else {
                const float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n0 + e < args.N) store_out_one<OT>(args.out, at + e, y[e]);
            }
        }
        if (clustered) {
            // no CTA leaves while another may still read its sums
            cluster_arrive();
            cluster_wait();
        }
    }
    if (clustered && warp < 3) {
        // one arrive / wait pair per thread for each of the two meetings above
        cluster_arrive();
        cluster_wait();
        cluster_arrive();
        cluster_wait();
    }
    // every read of the accumulators lies before this point
    tc_fence_before();
    __syncthreads();
    // whichever warp's wait ran out: the copies already issued land before the CTA can exit
    if (threadIdx.x == 0 && *abort_flag) drain_ring(full, L::STAGES, *issued);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L::TMEM_COLS);
    }
}

}  // namespace nvfp4lora
