// E4M3 x E4M3 product with fp32 scales per block of 128, tiled SM-pair kernel (sm_100a).
//
//     out[m, n] = round( sum_kb sa[m, kb] * sb[n / 128, kb] * P_kb[m, n]  [+ bias[n]] ),
//     P_kb[m, n] = sum over the 128 columns k of block kb of a[m, k] * b[n, k].
// The scales are general fp32 numbers, so they cannot ride on the tensor cores' own block scaling
// (powers of two, or e4m3): each P_kb is formed in TMEM by itself, read back and added to an fp32
// accumulator in registers, acc = fma(sa * sb, P_kb, acc).
//
// Scales and bias are read with plain loads after the dependency wait: read-only (nc) loads carry no ordering
// against it, and the compiler moved them ahead of it, where the kernel before was still writing them.
//
// A cluster of two CTAs computes one 256 x 256 output tile per step with tcgen05.mma.cta_group::2
// (kind::f8f6f4, M = 256, N = 256, K = 32): each CTA loads its own 128 rows of A and 128 of the
// tile's 256 B rows, 32 KB per CTA and K block, through a ring of six.  The TMEM holds two 256-column
// accumulators used in turn, so the MMAs of a K block (4 x 128 cycles) run while the eight promotion
// warps of each CTA read the previous one (128 lanes x 256 columns: one warp per lane quarter and 128
// columns, which see a single sb per K block).  Registers are split by warpgroup: the promotion warps
// hold 128 fp32 sums each and read 16 columns at a time (with 32 the loop spilled: 2.2 ms against 1.5 at
// 8192 x 28672 x 8192; 16 bytes of spills per thread are left with 16-bit outputs).
// With few tiles (TN = 128) a tile is 256 x 128, so that twice as many SM pairs work: four products of 128 columns in
// TMEM, 64 columns per promotion warp, no register split.
// What bounds it: the promotion, not the tensor pipe.  A K block takes about 850 cycles without operand loads and
// 950 to 1100 with them, against 512 of MMAs: a promotion warp needs about 410 for its 128 columns, 185 to see a
// product that is ready and 260 for the rest of its loop (the last two are latency, not a limit).  8192 x 28672 x 8192
// runs 1.55 to 1.68 ms in short runs (2.3 to 2.5 PFLOP/s, 0.67 to 0.72 of twice the measured bf16 rate) and 1.88 to
// 1.90 back to back (0.59 to 0.60), under the power limit.  Products of 128 columns (four in TMEM) with two
// issuers, sixteen promotion warps of 64 columns, scales staged by a warp of their own and scales loaded two to four
// blocks ahead all measured level or slower.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "ptx.cuh"

namespace nvfp4lora {

enum class OutType { BF16 = 0, FP16 = 1, FP32 = 2 };

struct Fp8GemmArgs {
    const float* a_scale;    // element (m, kb) at m * stride_am + kb * stride_ak
    const float* b_scale;    // [ceil(N / 128), kblocks] row-major
    const uint16_t* bias;    // bf16 [N] or null
    void* out;               // [M, N]
    int64_t stride_am, stride_ak;
    int M, N, kblocks;       // kblocks = ceil(K / 128)
    int m_tiles, n_tiles, num_tiles;
    int out_bytes;           // alignment of out's rows: 16 (TMA stores), 8, 4 or 2 bytes
};

// Instruction descriptor: kind::f8f6f4, E4M3 x E4M3 -> fp32, K-major A and B.
__host__ __device__ constexpr uint32_t idesc_e4m3_m(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void tc_mma_fp8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One K = 32 step of a single CTA's MMA (the split-K kernel).
__device__ __forceinline__ void tc_mma_fp8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// True in one lane of a converged warp.  A warp that issues MMAs runs its loop with all lanes and issues
// under this predicate: the compiler then keeps the descriptors in uniform registers.  Issued by
// `lane == 0` code each MMA waited for its operands to be moved there (about 70 cycles).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "elect.sync _|p, 0xffffffff;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Bounded wait whose try_wait carries no suspend-time hint: the hand-off of a K block's product passes
// through three of these, and with the 1 ms hint of mbar_wait each woke later (8192 x 28672 x 8192: 1556 us
// against 1504).  Polling with test_wait instead took issue slots from the promotion warps (1654 us).
__device__ __forceinline__ bool mbar_try_wait_short(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return done != 0;
}

__device__ __forceinline__ bool mbar_wait_short(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (mbar_try_wait_short(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait_short(bar, parity)) return true;
        if (abort != nullptr && *abort) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            if (abort != nullptr) *abort = 1;
            report_timeout();
            return false;
        }
    }
}

// {a.x, a.y} + s * {p.x, p.y}, each rounded to nearest even (one packed fma)
__device__ __forceinline__ void fma2(float& ax, float& ay, uint32_t px, uint32_t py, uint64_t ss) {
    uint64_t d;
    asm("{\n\t.reg .b64 pa, pp;\n\t"
        "mov.b64 pa, {%1, %2};\n\t"
        "mov.b64 pp, {%3, %4};\n\t"
        "fma.rn.f32x2 %0, pp, %5, pa;\n\t}"
        : "=l"(d) : "f"(ax), "f"(ay), "r"(px), "r"(py), "l"(ss));
    ax = __uint_as_float((uint32_t)d);
    ay = __uint_as_float((uint32_t)(d >> 32));
}

__device__ __forceinline__ uint64_t dup2(float s) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(s));
    return d;
}

// `out` values of one type, packed two (16-bit types) per word.
template <OutType OT>
__device__ __forceinline__ uint32_t pack_out2(float a, float b) {
    if constexpr (OT == OutType::FP16) {
        const __half2 h = __floats2half2_rn(a, b);
        uint32_t u;
        memcpy(&u, &h, 4);
        return u;
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        uint32_t u;
        memcpy(&u, &h, 4);
        return u;
    }
}

template <OutType OT>
__device__ __forceinline__ void store_out_one(void* out, int64_t i, float v) {
    if constexpr (OT == OutType::FP32) static_cast<float*>(out)[i] = v;
    else if constexpr (OT == OutType::FP16) static_cast<__half*>(out)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
}

constexpr int kFp8TileM = 256;           // per SM pair: 128 rows per CTA
constexpr int kFp8Threads = 384;         // warpgroup 0: producer, MMA issuer; 1 and 2: promotion
constexpr int kFp8EpiWarps = 8;
constexpr int kFp8BoxRows = 32;
// Registers per thread after the split: the block is launched with 384 x 168 and the shares must not
// exceed that pool (setmaxnreg.inc waits for registers that the other warpgroup gives back).
constexpr int kFp8RegsLaunch = 168;
constexpr int kFp8RegsCtl = 72;
constexpr int kFp8RegsEpi = 216;
static_assert(128 * kFp8RegsCtl + 256 * kFp8RegsEpi <= kFp8Threads * kFp8RegsLaunch,
              "register split exceeds the launch's register pool");

// TN: columns of a tile, 256 or 128.
template <int TN>
struct Fp8Smem {
    static constexpr int STAGES = TN == 256 ? 6 : 8;
    static constexpr int PRODUCTS = 512 / TN;             // products of a K block in TMEM
    static constexpr int A_BYTES = 128 * 128;
    static constexpr int B_BYTES = TN / 2 * 128;
    static constexpr int STAGE_TX = A_BYTES + B_BYTES;    // per CTA, on the leader's barrier
    static constexpr int A_OFF = 0;
    static constexpr int B_OFF = A_OFF + STAGES * A_BYTES;
    static constexpr int OUT_OFF = B_OFF + STAGES * B_BYTES;
    static constexpr int BOX_BYTES = 64 * kFp8BoxRows;    // 32 columns of a 16-bit type, 16 of fp32
    static constexpr int BAR_OFF = OUT_OFF + kFp8EpiWarps * 2 * BOX_BYTES;
    static constexpr int NUM_BARS = 2 * STAGES + 2 * PRODUCTS + 1;    // full, empty, acc_full, acc_empty, drain
    static constexpr int MISC_OFF = BAR_OFF + NUM_BARS * 8;
    static constexpr int TOTAL = MISC_OFF + 16;
    static constexpr int DYN_BYTES = TOTAL + 1024;
    static_assert(DYN_BYTES <= 232448, "shared-memory plan exceeds 227 KB");
};

// Tile order: bands of kFp8Band m tiles, m fastest within a band, so that the pairs running at one time
// share both operands' tiles (8192 x 4096 x 8192: 303 us, 371 with m fastest over the whole matrix; bands of 4, 6, 10,
// 12 and 16 within 5 %, none faster at every shape).
constexpr int kFp8Band = 8;

__device__ __forceinline__ void fp8_tile(int tile, int m_tiles, int n_tiles, int& m_blk, int& n_blk) {
    const int band = tile / (kFp8Band * n_tiles);
    const int r = tile - band * kFp8Band * n_tiles;
    const int bm = min(kFp8Band, m_tiles - band * kFp8Band);
    n_blk = r / bm;
    m_blk = band * kFp8Band + r - n_blk * bm;
}

// Byte `at` of row r in a box of 32 rows of 64 bytes.
__device__ __forceinline__ int fp8_box_at(int r, int at) { return r * 64 + (at ^ ((r >> 1 & 3) << 4)); }

// The part of a box that lies in out (rows x cols elements from `out` on), a vector V of its rows' alignment per lane
// (6606 x 21984 x 1472: 233 us with TMA stores; 278 to 328 with 4 bytes per lane at N = 21986, 359 to 380 with 2 at 21987;
// 300 x 4100 x 4112, 8 bytes: 15.1 us, 16.9 with one element per lane).
template <typename V, typename E>
__device__ __forceinline__ void fp8_store_box(const uint8_t* box, E* out, int64_t N, int rows, int cols, int lane) {
    constexpr int PER = 64 / (int)sizeof(V), STEP = 32 / PER;      // lanes per row, rows per step
    const int at = lane % PER * (int)sizeof(V), c = at / (int)sizeof(E);
    if (c >= cols) return;
#pragma unroll 4
    for (int r = lane / PER; r < 32; r += STEP)
        if (r < rows) *reinterpret_cast<V*>(out + r * N + c) = *reinterpret_cast<const V*>(box + fp8_box_at(r, at));
}

// The K block that a tile starts with; it goes on around the end.  Tiles that run at one time and share an operand
// would otherwise all read the same lines of it at the same time, from a few L2 slices (256 x 8192 x 8192: 37 us
// with every tile from block 0, 30 with this; 300 x 4100 x 4112: 19.6 and 17.1; large products are level).  The order
// of an element's sum so depends on its tile: equal rows of a in different row tiles may differ in their last bits, while
// a repeated call gives the same bits.
__device__ __forceinline__ int fp8_first_block(int m_blk, int n_blk, int kblocks) {
    return (int)((3u * (uint32_t)n_blk + (uint32_t)m_blk) % (uint32_t)kblocks);
}

template <OutType OT, int TN>
__global__ void __launch_bounds__(kFp8Threads, 1)
fp8_gemm_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_out, const Fp8GemmArgs args) {
    using L = Fp8Smem<TN>;
    constexpr uint32_t IDESC = idesc_e4m3_m(kFp8TileM, TN);
    constexpr uint16_t kBoth = 0x3;
    constexpr uint32_t kAll = 0xffffffffu;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);   // the leader's is used
    uint64_t* empty = full + L::STAGES;
    uint64_t* acc_full = empty + L::STAGES;        // a K block's product is complete
    uint64_t* acc_empty = acc_full + L::PRODUCTS;  // the leader's: both CTAs have read it
    uint64_t* drain = acc_empty + L::PRODUCTS;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC_OFF + 4);
    volatile uint32_t* issued = reinterpret_cast<volatile uint32_t*>(smem + L::MISC_OFF + 8);   // K blocks copied by this CTA

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();          // 0: the leader, which issues the MMAs
    const int pair = blockIdx.x >> 1;
    const int npairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        prefetch_tensor_map(&tm_a);
        prefetch_tensor_map(&tm_b);
        if (args.out_bytes == 16) prefetch_tensor_map(&tm_out);
        for (int s = 0; s < L::STAGES; ++s) {
            mbar_init(&full[s], 1);                // the leader's expect_tx; bytes from both CTAs
            mbar_init(&empty[s], 1);               // the leader's multicast commit
        }
        for (int k = 0; k < L::PRODUCTS; ++k) {
            mbar_init(&acc_full[k], 1);            // the leader's multicast commit
            mbar_init(&acc_empty[k], 2 * kFp8EpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // both CTAs' barriers exist before any copy completes on, or any thread arrives at, the peer
    cluster_arrive();
    cluster_wait();
    const uint32_t tmem = *tmem_slot;
    grid_launch_dependents();

    if (warp < 4) {
        if constexpr (TN == 256) reg_dealloc<kFp8RegsCtl>();
        if (warp == 0 && lane == 0) {
            // ------------------------------- TMA producer (both CTAs) -------------------------------
            grid_dependency_wait();
            int stage = 0;
            uint32_t phase = 0, n = 0;
            bool ok = true;
            for (int tile = pair; ok && tile < args.num_tiles; tile += npairs) {
                int m_blk, n_blk;
                fp8_tile(tile, args.m_tiles, args.n_tiles, m_blk, n_blk);
                const int row_a = m_blk * kFp8TileM + (int)rank * 128;   // this CTA's A rows
                const int row_b = n_blk * TN + (int)rank * (TN / 2);   // and B half
                int kx = fp8_first_block(m_blk, n_blk, args.kblocks);
                for (int kb = 0; kb < args.kblocks; ++kb, ++n) {
                    if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) { ok = false; break; }
                    const uint32_t lead_full = map_to_rank(smem_u32(&full[stage]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * L::STAGE_TX);
                    tma_load_2d_pair(smem + L::A_OFF + stage * L::A_BYTES, &tm_a, lead_full, kx * 128, row_a);
                    tma_load_2d_pair(smem + L::B_OFF + stage * L::B_BYTES, &tm_b, lead_full, kx * 128, row_b);
                    if (++kx == args.kblocks) kx = 0;
                    if (++stage == L::STAGES) { stage = 0; phase ^= 1; }
                }
            }
            *issued = n;
        } else if (warp == 1 && rank == 0) {
            // ------------------------------- MMA issuer (the leader) -------------------------------
            grid_dependency_wait();
            int stage = 0;
            uint32_t phase = 0, g = 0;             // g: K blocks issued so far, over all tiles
            bool ok = true;
            for (int tile = pair; ok && tile < args.num_tiles; tile += npairs) {
                for (int kb = 0; kb < args.kblocks; ++kb, ++g) {
                    const uint32_t buf = g % L::PRODUCTS;
                    ok = mbar_wait_short(&full[stage], phase, abort_flag) &&
                         mbar_wait_short(&acc_empty[buf], ((g / L::PRODUCTS) & 1) ^ 1, abort_flag);
                    if (!__all_sync(kAll, ok)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(smem + L::A_OFF + stage * L::A_BYTES);
                    const uint32_t b_addr = smem_u32(smem + L::B_OFF + stage * L::B_BYTES);
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            tc_mma_fp8_pair(tmem + buf * TN, sdesc_sw128(a_addr + j * 32),
                                            sdesc_sw128(b_addr + j * 32), IDESC, j > 0 ? 1u : 0u);
                        tc_commit_pair_multicast(&acc_full[buf], kBoth);
                        tc_commit_pair_multicast(&empty[stage], kBoth);
                    }
                    __syncwarp();
                    if (++stage == L::STAGES) { stage = 0; phase ^= 1; }
                }
            }
            if (!ok || *abort_flag) {
                // Wait for the MMAs already issued before TMEM is released.
                if (elect_one()) {
                    tc_commit_pair_multicast(drain, 0x1);
                    mbar_wait(drain, 0, nullptr);
                }
            }
        }
        __syncwarp();
    } else {
        if constexpr (TN == 256) reg_alloc<kFp8RegsEpi>();
        // ------------------------------- promotion and epilogue (both CTAs) -------------------------------
        const int ew = warp - 4;                       // 0..7
        const int q = warp & 3;                        // TMEM lane quarter of this warp
        const int h = ew >> 2;                         // which half of the tile's columns
        const uint32_t lane_off = (uint32_t)(q * 32) << 16;
        grid_dependency_wait();
        const uint32_t lead_acc_empty = map_to_rank(smem_u32(acc_empty), 0);
        uint32_t g = 0;
        bool ok = true;
        for (int tile = pair; ok && tile < args.num_tiles; tile += npairs) {
            int m_blk, n_blk;
            fp8_tile(tile, args.m_tiles, args.n_tiles, m_blk, n_blk);
            const int row0 = m_blk * kFp8TileM + (int)rank * 128 + q * 32;   // this warp's 32 rows
            const int col0 = n_blk * TN + h * (TN / 2);
            const float* sa = args.a_scale + (int64_t)min(row0 + lane, args.M - 1) * args.stride_am;
            const float* sb = args.b_scale + (int64_t)min(col0 / 128, (args.N - 1) / 128) * args.kblocks;
            float acc[TN / 2];
#pragma unroll
            for (int k = 0; k < TN / 2; ++k) acc[k] = 0.0f;
            // the scales of the next block, loaded one block ahead; they are multiplied when used (a multiply
            // here would stall the warp on the loads)
            int kx = fp8_first_block(m_blk, n_blk, args.kblocks);
            float sa_next = sa[kx * args.stride_ak], sb_next = sb[kx];
            for (int kb = 0; kb < args.kblocks; ++kb, ++g) {
                const uint32_t buf = g % L::PRODUCTS;
                const uint64_t ss = dup2(sa_next * sb_next);
                if (kb + 1 < args.kblocks) {
                    if (++kx == args.kblocks) kx = 0;
                    sa_next = sa[kx * args.stride_ak];
                    sb_next = sb[kx];
                }
                if (!__all_sync(kAll, mbar_wait_short(&acc_full[buf], (g / L::PRODUCTS) & 1, abort_flag))) { ok = false; break; }
                tc_fence_after();
                const uint32_t src = tmem + lane_off + buf * TN + h * (TN / 2);
                uint32_t p[2][16];
                tmem_load_16(src, p[0]);
#pragma unroll
                for (int c = 0; c < TN / 32; ++c) {
                    tmem_load_wait();
                    if (c < TN / 32 - 1) tmem_load_16(src + 16 * (c + 1), p[(c + 1) & 1]);
                    else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote_relaxed(lead_acc_empty + buf * 8);
                    }
#pragma unroll
                    for (int k = 0; k < 16; k += 2) fma2(acc[c * 16 + k], acc[c * 16 + k + 1], p[c & 1][k], p[c & 1][k + 1], ss);
                }
            }
            if (!ok) break;
            // 64 bytes of each of the warp's 32 rows at a time through its two boxes in shared memory, in turn.  The
            // 16-byte parts of a row are swizzled by its number (SWIZZLE_64B), so that eight lanes' rows meet no
            // bank twice.
            using E = typename std::conditional<OT == OutType::FP32, uint32_t, uint16_t>::type;
            constexpr int COLS = 64 / (int)sizeof(E);
            if (args.out_bytes == 16 && lane == 0) bulk_wait_group_read<0>();   // the last tile's stores have read the boxes
            if (args.bias != nullptr) {
                // through the boxes, so that a thread reads four columns' values at a time
                __syncwarp();
                float* bias = reinterpret_cast<float*>(smem + L::OUT_OFF + ew * 2 * L::BOX_BYTES);
                uint32_t raw[TN / 64];                 // all loads before the first store
#pragma unroll
                for (int k = 0; k < TN / 64; ++k) raw[k] = args.bias[min(col0 + k * 32 + lane, args.N - 1)];
#pragma unroll
                for (int k = 0; k < TN / 64; ++k) bias[k * 32 + lane] = __uint_as_float(raw[k] << 16);
                __syncwarp();
#pragma unroll
                for (int k = 0; k < TN / 2; k += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(bias + k);
                    acc[k] = __fadd_rn(acc[k], v.x);
                    acc[k + 1] = __fadd_rn(acc[k + 1], v.y);
                    acc[k + 2] = __fadd_rn(acc[k + 2], v.z);
                    acc[k + 3] = __fadd_rn(acc[k + 3], v.w);
                }
            }
#pragma unroll
            for (int x = 0; x < TN / 2; x += COLS) {
                if (col0 + x >= args.N || row0 >= args.M) break;
                uint8_t* box = smem + L::OUT_OFF + (ew * 2 + (x / COLS) % 2) * L::BOX_BYTES;
                if (x > 0 && args.out_bytes == 16 && lane == 0) bulk_wait_group_read<1>();   // the box's previous store has read it
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float* v = acc + x + k * (COLS / 4);
                    uint4* dst = reinterpret_cast<uint4*>(box + fp8_box_at(lane, k * 16));
                    if constexpr (OT == OutType::FP32)
                        *dst = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                          __float_as_uint(v[3]));
                    else
                        *dst = make_uint4(pack_out2<OT>(v[0], v[1]), pack_out2<OT>(v[2], v[3]),
                                          pack_out2<OT>(v[4], v[5]), pack_out2<OT>(v[6], v[7]));
                }
                if (args.out_bytes == 16) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&tm_out, box, col0 + x, row0);
                        bulk_commit_group();
                    }
                } else {
                    // rows of out off their 16-byte boundaries: neighbouring lanes store neighbouring columns
                    __syncwarp();
                    E* out = static_cast<E*>(args.out) + (int64_t)row0 * args.N + col0 + x;
                    const int rows = args.M - row0, cols = args.N - col0 - x;
                    if (args.out_bytes == 8) fp8_store_box<uint2>(box, out, args.N, rows, cols, lane);
                    else if (args.out_bytes == 4) fp8_store_box<uint32_t>(box, out, args.N, rows, cols, lane);
                    else if constexpr (sizeof(E) == 2) fp8_store_box<uint16_t>(box, out, args.N, rows, cols, lane);
                }
            }
        }
        if (args.out_bytes == 16 && lane == 0) bulk_wait_group_all();
    }

    tc_fence_before();
    pair_finish(full, L::STAGES, issued, abort_flag);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

}  // namespace nvfp4lora
