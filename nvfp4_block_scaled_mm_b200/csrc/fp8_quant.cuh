// E4M3 values with an fp32 scale per group of 128: the quantizer and the fused residual addition,
// root-mean-square norm and quantizer that make the 8-bit product's operands (sm_100a).
//
// For a group of values y (1 x 128 along a row, or a block of 128 x 128):
//     amax = max(max |y|, 2^-100);   scale = amax / 448;   q = E4M3_rne(y * (448 / amax))
// (448 is E4M3's largest finite value; the bound 2^-100 keeps the scale and its inverse normal
// numbers, and gives a group of zeros +-0 codes).  The norm's y is
//     h = x + residual;   residual <- round(h);   y = h * (1 / sqrt(mean(h^2) + eps)) * weight,
// all in fp32: the sum of squares, y and the group maxima come from the unrounded h, so that q is
// the only rounding to fewer bits on its path.
// A NaN stays a NaN in q and is ignored by amax; an infinity makes its group's scale infinite, itself a NaN and
// the group's finite values zeros.  In the norm an infinity, or finite values whose mean square passes fp32's range,
// make rms zero: zeros, and a NaN in an infinity's place.
//
// HBM-bound: the norm of 8192 x 8192 bf16 with residual and the normed rows kept runs 92 us (6.6 TB/s), of 65536 x 512
// 36 us (6.5); without either, where it moves 3 bytes per element, 45 us (4.5), at two thirds of the issue slots and of the
// copy rate: a row's loads, the barrier and the arithmetic follow each other within a CTA.
// The quantizer of 8192 x 8192 takes 32 us by rows (6.3) and of 28672 x 8192 102 us by blocks (6.9, part of the
// writes still in L2).  Sixteen rows take 2 us, launch latency.  Rows off 16 bytes take element accesses: the norm of 883 x
// 5804 14.7 us (6.3 at 5808), the quantizer of 11805 x 4570 53 (27 at 4576).
#pragma once

#include <cstdint>

#include "moe.cuh"
#include "ptx.cuh"
#include "quantize.cuh"

namespace nvfp4lora {

constexpr int kNormMaxThreads = 512;     // NV = 4 holds a row of 16384 elements
constexpr float kFp8Max = 448.0f;
constexpr float kFp8Tiny = 0x1p-100f;

struct Fp8QuantArgs {
    const void* x;           // [rows, H]
    void* residual;          // [rows, H] or null (norm only)
    const void* weight;      // [H] (norm only)
    void* norm_out;          // [rows, H] or null (norm only)
    uint8_t* q;              // [rows, H]
    float* scales;           // element (r, g) at r * stride_r + g * stride_g
    int64_t stride_r, stride_g;
    int64_t rows, H;
    float eps;
};

// two float32 -> two E4M3 bytes, `a` in the low one (nearest even, saturating; NaN stays NaN)
__device__ __forceinline__ uint32_t e4m3x2_rn(float a, float b) {
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(b), "f"(a));
    return two;
}

// Packed fp32 arithmetic on eight values, each operation rounded to nearest even: half the instructions (the norm
// is bound by instruction issue where it moves few bytes).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ float2 unpack2(uint64_t d) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(d));
    return v;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t fma2_rn(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ uint2 e4m3x8_scaled(const float (&y)[8], float inv) {
    const uint64_t s = pack2(inv, inv);
    uint32_t two[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = unpack2(mul2(pack2(y[2 * i], y[2 * i + 1]), s));
        two[i] = e4m3x2_rn(v.x, v.y);
    }
    return make_uint2(two[0] | (two[1] << 16), two[2] | (two[3] << 16));
}

__device__ __forceinline__ float abs_max8(const float (&y)[8]) {
    float m = fmaxf(fabsf(y[0]), fabsf(y[1]));
#pragma unroll
    for (int i = 2; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
    return m;
}

// Maxima of pairs of 16-bit values: the larger magnitude of a group is one of its values, so nothing is rounded, and
// two rows' maxima are shuffled as one word.  A NaN is ignored, as by fmaxf.
template <MoeType TY>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (TY == MoeType::BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Largest magnitudes of the even (low half) and the odd of eight 16-bit values.
template <MoeType TY>
__device__ __forceinline__ uint32_t abs_max_pairs(const uint4& w) {
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    return max2<TY>(max2<TY>(w.x & kAbs, w.y & kAbs), max2<TY>(w.z & kAbs, w.w & kAbs));
}

template <MoeType TY>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
    return to_f32<TY>(static_cast<const typename MoeElem<TY>::type*>(p)[i]);
}

template <MoeType TY>
__device__ __forceinline__ void store_one(void* p, int64_t i, float y) {
    static_cast<typename MoeElem<TY>::type*>(p)[i] = from_f32<TY>(y);
}

// Sum over the CTA, the same in every thread (fixed order).  `red` holds 32 floats.
__device__ __forceinline__ float cta_sum(float s, float* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (blockDim.x + 31) >> 5;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    if (lane == 0) red[warp] = s;
    __syncthreads();
    float t = lane < nw ? red[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, d);
    return t;
}

// ---- norm: the row kept in registers (NV chunks of 256 elements per warp); a CTA per row, or, with SHORT, a warp
// per row of up to 1024 elements ----
// HBM-bound: 2 + 1 bytes per element (16-bit types), and 4 more with a residual.  A chunk is two 1 x 128
// groups: with VEC (aligned rows, H % 8 == 0) one per half-warp, otherwise the lanes' first and last four.
constexpr int kNormShortRows = 8;          // rows (warps) of a SHORT CTA

template <MoeType TY, int NV, bool VEC, bool SHORT>
__global__ void __launch_bounds__(kNormMaxThreads, SHORT || !VEC ? 0 : NV == 4 ? 2 : NV == 1 && TY != MoeType::FP32 ? 4 : 0)
rmsnorm_fp8_kernel(const Fp8QuantArgs a) {
    using C = RowChunk<TY, VEC, VEC>;          // with VEC, H % 8 == 0
    __shared__ float red[32];
    const int lane = threadIdx.x & 31, warp = SHORT ? 0 : threadIdx.x >> 5, nw = SHORT ? 1 : blockDim.x >> 5;
    const int64_t row = SHORT ? (int64_t)blockIdx.x * kNormShortRows + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    const int64_t H = a.H;
    if (SHORT && row >= a.rows) return;        // no barrier follows
    const void* x = row_at<TY>(a.x, row, H);
    void* res = a.residual != nullptr ? row_at<TY>(a.residual, row, H) : nullptr;
    float h[NV][8];
    // rows of four chunks per warp load the weight after the sum: held across it, it would spill at the 64
    // registers of two CTAs of 512 threads (fp32 rows spill 60 bytes as it is)
    constexpr bool kLate = NV == 4;
    typename C::Raw wt[kLate ? 1 : NV];
    grid_dependency_wait();
    grid_launch_dependents();
    uint64_t ss2 = 0;                          // the even and the odd elements' sums
    {
        typename C::Raw xr[NV], rr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t e0 = (int64_t)(warp + i * nw) * 256;
            xr[i] = C::load(x, e0, H, lane);
            if (res != nullptr) rr[i] = C::load(res, e0, H, lane);
            if constexpr (!kLate) wt[i] = C::load(a.weight, e0, H, lane);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            C::unpack(xr[i], h[i]);
            if (res != nullptr) {
                float r[8];
                C::unpack(rr[i], r);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] += r[e];
                C::store(res, (int64_t)(warp + i * nw) * 256, H, lane, h[i]);
            }
#pragma unroll
            for (int e = 0; e < 8; e += 2) {   // elements past H are 0
                const uint64_t v = pack2(h[i][e], h[i][e + 1]);
                ss2 = fma2_rn(v, v, ss2);
            }
        }
    }
    float ss = unpack2(ss2).x + unpack2(ss2).y;
    if constexpr (SHORT) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
    } else {
        ss = cta_sum(ss, red);
    }
    const float rms = rsqrtf(ss / (float)H + a.eps);
    float* sc = a.scales + row * a.stride_r;
    uint8_t* q = a.q + row * H;
    const uint64_t rms2 = pack2(rms, rms);
    float mine = 1.0f;                         // VEC: lane i of a half-warp divides for its group of chunk i
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t e0 = (int64_t)(warp + i * nw) * 256;
        float(&y)[8] = h[i];
        float w[8];
        if constexpr (!kLate) C::unpack(wt[i], w);
        else C::unpack(C::load(a.weight, e0, H, lane), w);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 v = unpack2(mul2(mul2(pack2(y[e], y[e + 1]), rms2), pack2(w[e], w[e + 1])));
            y[e] = v.x;
            y[e + 1] = v.y;
        }
        if constexpr (VEC) {
            float m = abs_max8(y);
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
            if (NV == 1 || (lane & 15) == i) mine = fmaxf(m, kFp8Tiny);
        } else {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                float m = fmaxf(fmaxf(fabsf(y[4 * g]), fabsf(y[4 * g + 1])), fmaxf(fabsf(y[4 * g + 2]), fabsf(y[4 * g + 3])));
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
                m = fmaxf(m, kFp8Tiny);
                const float inv = __fdiv_rn(kFp8Max, m);
#pragma unroll
                for (int e = 4 * g; e < 4 * g + 4; ++e)
                    if (C::at(e0, lane, e) < H) q[C::at(e0, lane, e)] = (uint8_t)e4m3x2_rn(y[e] * inv, 0.0f);
                if (lane == 0 && e0 + g * 128 < H) sc[(e0 / 128 + g) * a.stride_g] = __fdiv_rn(m, kFp8Max);
            }
        }
        if (a.norm_out != nullptr) C::store(row_at<TY>(a.norm_out, row, H), e0, H, lane, y);
    }
    if constexpr (VEC) {
        const float inv_mine = __fdiv_rn(kFp8Max, mine);
        const int64_t g = (int64_t)(warp + (lane & 15) * nw) * 2 + (lane >> 4);
        if ((lane & 15) < NV && g * 128 < H) sc[g * a.stride_g] = __fdiv_rn(mine, kFp8Max);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float inv = NV == 1 ? inv_mine : __shfl_sync(0xFFFFFFFFu, inv_mine, (lane & 16) + i);
            const int64_t at = (int64_t)(warp + i * nw) * 256 + lane * 8;
            if (at < H) *reinterpret_cast<uint2*>(q + at) = e4m3x8_scaled(h[i], inv);
        }
    }
}

// ---- a CTA per row, a warp per group, any row length and alignment ----
// NORM = false: the quantizer of x itself.  NORM = true: the norm of rows longer than a CTA's registers hold,
// which are read twice.
template <MoeType TY, bool NORM>
__global__ void __launch_bounds__(256)
row_fp8_kernel(const Fp8QuantArgs a) {
    __shared__ float red[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int64_t base = (int64_t)blockIdx.x * a.H;
    grid_dependency_wait();
    grid_launch_dependents();
    auto load_h = [&](int64_t i) {
        float h = load_one<TY>(a.x, base + i);
        if (NORM && a.residual != nullptr) h += load_one<TY>(a.residual, base + i);
        return h;
    };
    float rms = 1.0f;
    if (NORM) {
        float ss = 0.0f;
        for (int64_t i = threadIdx.x; i < a.H; i += blockDim.x) {
            const float h = load_h(i);
            ss = fmaf(h, h, ss);
        }
        rms = rsqrtf(cta_sum(ss, red) / (float)a.H + a.eps);
    }
    const int H = (int)a.H, groups = (H + 127) / 128;
    // Groups per warp at a time, their loads first and one division for all: 300 x 40001 normed 70 us with four, 100
    // with one; without the norm's loads two are slower (11805 x 4570 60 us, 54 with one).
    constexpr int NG = NORM ? 4 : 1;
    for (int g0 = warp * NG; g0 < groups; g0 += nw * NG) {
        float y[NG][4], mine = 1.0f;           // lane i divides for group g0 + i
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = (g0 + i) * 128 + e * 32 + lane;
                y[i][e] = c < H ? load_h(c) : 0.0f;
            }
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = (g0 + i) * 128 + e * 32 + lane;
                if (NORM && c < H) {
                    if (a.residual != nullptr) store_one<TY>(a.residual, base + c, y[i][e]);
                    y[i][e] = y[i][e] * rms * load_one<TY>(a.weight, c);
                    if (a.norm_out != nullptr) store_one<TY>(a.norm_out, base + c, y[i][e]);
                }
                m = fmaxf(m, fabsf(y[i][e]));
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
            if (NG == 1 || lane == i) mine = fmaxf(m, kFp8Tiny);
        }
        const float inv_mine = __fdiv_rn(kFp8Max, mine);
        if (lane < NG && g0 + lane < groups)
            a.scales[blockIdx.x * a.stride_r + (g0 + lane) * a.stride_g] = __fdiv_rn(mine, kFp8Max);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const float inv = NG == 1 ? inv_mine : __shfl_sync(0xFFFFFFFFu, inv_mine, i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = (g0 + i) * 128 + e * 32 + lane;
                if (c < H) a.q[base + c] = (uint8_t)e4m3x2_rn(y[i][e] * inv, 0.0f);
            }
        }
    }
}

// ---- quantizer of aligned rows (H % 8 == 0): a CTA per 128 rows x 128 columns, kept in registers ----
// HBM-bound: 2 bytes read (16-bit types) and 1 written per element.  Sixteen lanes hold 128 columns of a row, each
// thread 8 rows of 8 columns, all loaded before the first is used.  BLOCK: one scale for the tile, otherwise one per
// row.
template <MoeType TY, bool BLOCK>
__global__ void __launch_bounds__(256)
quantize_fp8_tile_kernel(const Fp8QuantArgs a) {
    using R = RowChunk<TY, true, true>;
    __shared__ float red[8];
    const int nv = (int)(a.H / 8);
    const int64_t gcols = (a.H + 127) / 128;
    const int64_t br = blockIdx.x / gcols, bc = blockIdx.x % gcols;
    const int c = (int)bc * 16 + (threadIdx.x & 15);
    const int64_t r0 = br * 128 + (threadIdx.x >> 4);
    grid_dependency_wait();
    grid_launch_dependents();
    typename R::Raw raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c < nv && r0 + i * 16 < a.rows) raw[i] = R::load(a.x, ((r0 + i * 16) * nv + c) * 8, INT64_MAX, 0);
    if constexpr (BLOCK) {
        float m = 0.0f;
        if constexpr (TY == MoeType::FP32) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c < nv && r0 + i * 16 < a.rows) m = fmaxf(m, abs_max8(raw[i].e));
        } else {
            uint32_t m2 = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c < nv && r0 + i * 16 < a.rows) m2 = max2<TY>(m2, abs_max_pairs<TY>(raw[i].w[0]));
            m = fmaxf(to_f32<TY>((uint16_t)m2), to_f32<TY>((uint16_t)(m2 >> 16)));
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
        __syncthreads();
        m = kFp8Tiny;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w]);
        const float inv = __fdiv_rn(kFp8Max, m);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c < nv && r0 + i * 16 < a.rows) {
                float y[8];
                R::unpack(raw[i], y);
                reinterpret_cast<uint2*>(a.q)[(r0 + i * 16) * nv + c] = e4m3x8_scaled(y, inv);
            }
        if (threadIdx.x == 0) a.scales[br * a.stride_r + bc * a.stride_g] = __fdiv_rn(m, kFp8Max);
    } else {
        // lane i of the sixteen divides for row i, once for all of them
        const int lane = threadIdx.x & 31, hl = threadIdx.x & 15;
        float mine = 1.0f;
        if constexpr (TY == MoeType::FP32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float m = c < nv && r0 + i * 16 < a.rows ? abs_max8(raw[i].e) : 0.0f;
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
                if (hl == i) mine = fmaxf(m, kFp8Tiny);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const uint32_t u = c < nv && r0 + i * 16 < a.rows ? abs_max_pairs<TY>(raw[i].w[0]) : 0u;
                const uint32_t v = c < nv && r0 + (i + 1) * 16 < a.rows ? abs_max_pairs<TY>(raw[i + 1].w[0]) : 0u;
                // row i in the low half, row i + 1 in the high
                uint32_t m2 = max2<TY>(__byte_perm(u, v, 0x5410), __byte_perm(u, v, 0x7632));
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) m2 = max2<TY>(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, d));
                if ((hl & ~1) == i) mine = fmaxf(to_f32<TY>((uint16_t)(hl & 1 ? m2 >> 16 : m2)), kFp8Tiny);
            }
        }
        const float inv_mine = __fdiv_rn(kFp8Max, mine);
        if (hl < 8 && r0 + hl * 16 < a.rows) a.scales[(r0 + hl * 16) * a.stride_r + bc * a.stride_g] = __fdiv_rn(mine, kFp8Max);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float inv = __shfl_sync(0xFFFFFFFFu, inv_mine, (lane & 16) + i);
            if (c < nv && r0 + i * 16 < a.rows) {
                float y[8];
                R::unpack(raw[i], y);
                reinterpret_cast<uint2*>(a.q)[(r0 + i * 16) * nv + c] = e4m3x8_scaled(y, inv);
            }
        }
    }
}

// ---- 128 x 128 blocks of any row length and alignment: a CTA per block, read twice ----
template <MoeType TY>
__global__ void __launch_bounds__(256)
blocks_fp8_kernel(const Fp8QuantArgs a) {
    __shared__ float red[8];
    const int64_t gcols = (a.H + 127) / 128;
    const int64_t br = blockIdx.x / gcols, bc = blockIdx.x % gcols;
    const int64_t c = bc * 128 + (threadIdx.x & 127);
    const int64_t r0 = br * 128 + (threadIdx.x >> 7), r1 = min(a.rows, br * 128 + 128);
    grid_dependency_wait();
    grid_launch_dependents();
    float m = 0.0f;
    if (c < a.H)
#pragma unroll 8
        for (int64_t r = r0; r < r1; r += 2) m = fmaxf(m, fabsf(load_one<TY>(a.x, r * a.H + c)));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    m = kFp8Tiny;
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w]);
    const float inv = __fdiv_rn(kFp8Max, m);
    if (c < a.H)
#pragma unroll 8
        for (int64_t r = r0; r < r1; r += 2)
            a.q[r * a.H + c] = (uint8_t)e4m3x2_rn(load_one<TY>(a.x, r * a.H + c) * inv, 0.0f);
    if (threadIdx.x == 0) a.scales[br * a.stride_r + bc * a.stride_g] = __fdiv_rn(m, kFp8Max);
}

}  // namespace nvfp4lora
