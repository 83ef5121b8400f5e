// Routed tokens: rows sorted by expert for the grouped call and back (sm_100a).
//
// With n = T * top_k slots, slot i = t * top_k + j of expert e_i = topk_ids[t, j] (active when
// 0 <= e_i < E), c_e the number of active slots of expert e and A the segment alignment:
//     m_indptr[0] = 0,  m_indptr[e + 1] = m_indptr[e] + A * ceil(c_e / A)
//     row(i) = m_indptr[e_i] + #{ i' < i : e_i' = e_i }   (-1 for an inactive slot)
//     rows[row(i)] = x[t];  slot_of[row(i)] = i, -1 for every other row.
// These are the m_indptr of the grouped call and the expanded_idx_to_permuted_idx of the LoRA
// delta (flashinfer.grouped_mm.grouped_mm_bf16, Parameters: m_indptr;
// flashinfer.fused_moe.bgmv_moe_gemm2_lora_delta, Parameters).  The order within an expert is the
// slot order, so the result does not depend on the schedule.
// Back: out[t] = sum_j w[t, j] * y[row(t, j)], and its gradients
//     gy[row(t, j)] = w[t, j] * g[t],   gw[t, j] = <g[t], y[row(t, j)]>;
// the gradient of the sorting is the sum without weights.  Sums are formed in fp32 in slot order
// (gw: a fixed tree over the row) and rounded once.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"

namespace nvfp4lora {

constexpr int kMoeThreads = 256;
constexpr int kMoeMaxTopK = 16;
constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxAlign = 4096;
constexpr int kMoeBatchSlots = 512;      // slots ranked at a time by one CTA (kMoeMaxTopK at least)
constexpr int kMoeCountChunks = 64;      // CTAs of the counting kernel
constexpr int kErrBadSlot = 4;           // device error word: an expert id or row index out of range

struct PermuteArgs {
    const uint8_t* x;        // [T] rows of row_bytes
    const int32_t* ids;      // [T, top_k]
    uint8_t* rows;           // [capacity] rows of row_bytes
    int32_t* indptr;         // [E + 1]
    int32_t* idx;            // [T * top_k]: slot -> row
    int32_t* inv;            // [capacity]: row -> slot
    const int32_t* counts;   // [kMoeCountChunks, E] slots per expert and chunk, or null: counted here
    int64_t chunk;           // slots per counting chunk
    int64_t n;               // T * top_k
    int64_t row_bytes;
    int T, top_k, E, align, capacity, zero_padding;
};

// Slots per expert of one chunk of the slots; a CTA per chunk.
__global__ void __launch_bounds__(kMoeThreads)
moe_count_kernel(const int32_t* __restrict__ ids, int64_t n, int64_t chunk, int E, int32_t* __restrict__ counts) {
    __shared__ int32_t hist[kMoeMaxExperts];
    for (int e = threadIdx.x; e < E; e += kMoeThreads) hist[e] = 0;
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t i0 = blockIdx.x * chunk, i1 = min(n, i0 + chunk);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kMoeThreads) {
        const int e = ids[i];
        if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kMoeThreads) counts[(int64_t)blockIdx.x * E + e] = hist[e];
}

template <int BYTES> struct MoeVec;
template <> struct MoeVec<16> { using type = uint4; };
template <> struct MoeVec<4> { using type = uint32_t; };
template <> struct MoeVec<2> { using type = uint16_t; };
template <> struct MoeVec<1> { using type = uint8_t; };

// Exclusive prefix sums over the experts of the aligned segment sizes (offs) and of the padding
// row counts (pads); offs[E] and pads[E] are the totals.  All threads of the CTA take part.
__device__ __forceinline__ void moe_scan(const int32_t* total, int E, int align, int32_t* offs, int32_t* pads) {
    __shared__ int32_t warp_seg[kMoeThreads / 32], warp_pad[kMoeThreads / 32];
    constexpr int PER = kMoeMaxExperts / kMoeThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t seg[PER], pad[PER], s = 0, p = 0;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int e = tid * PER + q;
        const int32_t c = e < E ? total[e] : 0;
        seg[q] = s;
        pad[q] = p;
        const int32_t a = (c + align - 1) / align * align;
        s += a;
        p += a - c;
    }
    int32_t is = s, ip = p;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t us = __shfl_up_sync(0xFFFFFFFFu, is, d), up = __shfl_up_sync(0xFFFFFFFFu, ip, d);
        if (lane >= d) { is += us; ip += up; }
    }
    if (lane == 31) { warp_seg[warp] = is; warp_pad[warp] = ip; }
    __syncthreads();
    int32_t bs = is - s, bp = ip - p;
    for (int w = 0; w < warp; ++w) { bs += warp_seg[w]; bp += warp_pad[w]; }
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int e = tid * PER + q;
        if (e <= E) { offs[e] = bs + seg[q]; pads[e] = bp + pad[q]; }
    }
    // E = kMoeMaxExperts: entry E lies past the last thread's experts
    if (tid == kMoeThreads - 1 && E == kMoeMaxExperts) { offs[E] = bs + s; pads[E] = bp + p; }
    __syncthreads();
}

// CTA c owns the tokens [T c / grid, T (c + 1) / grid).  It counts the slots of every expert before
// its own and in all (from the slots, or from the counting kernel's table plus the part of its own
// chunk), ranks its slots in order, and copies each of its tokens' rows to the token's up to top_k
// places, read once.  Padding rows and the row -> slot table's -1 entries are shared out evenly.
template <int VB>
__global__ void __launch_bounds__(kMoeThreads)
moe_permute_kernel(const PermuteArgs a) {
    using V = typename MoeVec<VB>::type;
    constexpr int UN = 4;                                   // vectors per lane and unit of copying
    __shared__ int32_t before[kMoeMaxExperts];              // slots of the expert before the next one ranked
    __shared__ int32_t total[kMoeMaxExperts];
    __shared__ int32_t offs[kMoeMaxExperts + 1];
    __shared__ int32_t pads[kMoeMaxExperts + 1];
    __shared__ int32_t place[kMoeBatchSlots];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = a.E, k = a.top_k;
    for (int e = tid; e < E; e += kMoeThreads) { before[e] = 0; total[e] = 0; }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();

    const int t0 = (int)((int64_t)a.T * blockIdx.x / gridDim.x);
    const int t1 = (int)((int64_t)a.T * (blockIdx.x + 1) / gridDim.x);
    const int64_t start = (int64_t)t0 * k;
    if (a.counts == nullptr) {
        // total[] holds the slots from `start` on until the two are added below
        for (int64_t i = tid; i < a.n; i += kMoeThreads) {
            const int e = a.ids[i];
            if (e >= 0 && e < E) atomicAdd(i < start ? &before[e] : &total[e], 1);
            else if (e >= E && blockIdx.x == 0) atomicExch(&g_device_error, kErrBadSlot);
        }
        __syncthreads();
        for (int e = tid; e < E; e += kMoeThreads) total[e] += before[e];
    } else {
        const int own = (int)(start / a.chunk);             // chunks before this one lie before `start`
        for (int e = tid; e < E; e += kMoeThreads) {
            int32_t b = 0, all = 0;
            for (int c = 0; c < kMoeCountChunks; ++c) {
                const int32_t v = a.counts[(int64_t)c * E + e];
                all += v;
                if (c < own) b += v;
            }
            before[e] = b;
            total[e] = all;
        }
        __syncthreads();
        for (int64_t i = own * a.chunk + tid; i < start; i += kMoeThreads) {
            const int e = a.ids[i];
            if (e >= 0 && e < E) atomicAdd(&before[e], 1);
        }
    }
    __syncthreads();
    moe_scan(total, E, a.align, offs, pads);
    if (blockIdx.x == 0)
        for (int e = tid; e <= E; e += kMoeThreads) a.indptr[e] = offs[e];

    // ---- this CTA's tokens, some at a time: rank their slots, then copy their rows ----
    const int64_t nv = a.row_bytes / VB;
    const int segs = (int)((nv + 32 * UN - 1) / (32 * UN));
    const int batch = kMoeBatchSlots / k;
    for (int tb = t0; tb < t1; tb += batch) {
        const int nt = min(batch, t1 - tb);
        if (warp == 0) {
            for (int s = 0; s < nt * k; s += 32) {
                const int64_t i = (int64_t)tb * k + s + lane;
                const bool in = s + lane < nt * k;
                int e = in ? a.ids[i] : -1;
                if (e >= E) {
                    if (a.counts != nullptr) atomicExch(&g_device_error, kErrBadSlot);
                    e = -1;
                }
                const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
                int32_t row = -1;
                if (e >= 0) row = offs[e] + before[e] + __popc(same & ((1u << lane) - 1u));
                __syncwarp();
                if (e >= 0 && lane == __ffs(same) - 1) before[e] += __popc(same);
                __syncwarp();
                if (in) {
                    place[s + lane] = row;
                    a.idx[i] = row;
                    if (row >= 0) a.inv[row] = (int32_t)i;
                }
            }
        }
        __syncthreads();
        for (int u = warp; u < nt * segs; u += kMoeThreads / 32) {
            const int t = u / segs, sg = u % segs;
            const V* src = reinterpret_cast<const V*>(a.x + (int64_t)(tb + t) * a.row_bytes) + (int64_t)sg * 32 * UN;
            const int64_t left = nv - (int64_t)sg * 32 * UN;
            V v[UN];
#pragma unroll
            for (int q = 0; q < UN; ++q)
                if (q * 32 + lane < left) v[q] = src[q * 32 + lane];
            for (int j = 0; j < k; ++j) {
                const int32_t row = place[t * k + j];
                if (row < 0) continue;
                V* dst = reinterpret_cast<V*>(a.rows + (int64_t)row * a.row_bytes) + (int64_t)sg * 32 * UN;
#pragma unroll
                for (int q = 0; q < UN; ++q)
                    if (q * 32 + lane < left) dst[q * 32 + lane] = v[q];
            }
        }
        __syncthreads();
    }

    // ---- padding rows, and the -1 entries of the row -> slot table ----
    const int npad = pads[E];
    const int gw = blockIdx.x * (kMoeThreads / 32) + warp, nw = gridDim.x * (kMoeThreads / 32);
    for (int p = gw; p < npad; p += nw) {
        int lo = 0, hi = E - 1;                             // the last expert with pads[e] <= p
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pads[mid] <= p) lo = mid; else hi = mid - 1;
        }
        const int row = offs[lo] + total[lo] + (p - pads[lo]);
        if (lane == 0) a.inv[row] = -1;
        if (a.zero_padding) {
            V* dst = reinterpret_cast<V*>(a.rows + (int64_t)row * a.row_bytes);
            for (int64_t q = lane; q < nv; q += 32) dst[q] = V{};
        }
    }
    for (int64_t r = (int64_t)offs[E] + blockIdx.x * kMoeThreads + tid; r < a.capacity; r += gridDim.x * kMoeThreads)
        a.inv[r] = -1;
}

// ---------------------------------------------------------------------------------------
// back: the weighted sum of a token's rows
// ---------------------------------------------------------------------------------------

enum class MoeType { BF16, FP16, FP32 };

// VE elements of one type: loaded together, as fp32, and rounded back (nearest, ties to even).
template <MoeType TY, int VE>
struct MoePack {
    static constexpr int ES = TY == MoeType::FP32 ? 4 : 2;
    using V = typename MoeVec<ES * VE>::type;
    static __device__ __forceinline__ void load(const void* p, int64_t i, float (&f)[VE]) {
        unpack(reinterpret_cast<const V*>(p)[i], f);
    }
    static __device__ __forceinline__ void unpack(const V& v, float (&f)[VE]) {
        if constexpr (TY == MoeType::FP32) {
            memcpy(f, &v, sizeof(v));
        } else {
            uint16_t h[VE];
            memcpy(h, &v, sizeof(v));
#pragma unroll
            for (int q = 0; q < VE; ++q)
                f[q] = TY == MoeType::BF16 ? __uint_as_float((uint32_t)h[q] << 16) : __half2float(__ushort_as_half(h[q]));
        }
    }
    static __device__ __forceinline__ V pack(const float (&f)[VE]) {
        V v;
        if constexpr (TY == MoeType::FP32) {
            memcpy(&v, f, sizeof(v));
        } else {
            uint16_t h[VE];
#pragma unroll
            for (int q = 0; q < VE; ++q)
                h[q] = TY == MoeType::BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f[q]))
                                           : __half_as_ushort(__float2half_rn(f[q]));
            memcpy(&v, h, sizeof(v));
        }
        return v;
    }
};

struct UnpermuteArgs {
    const void* y;           // [rows, H]
    const int32_t* idx;      // [T, top_k]: slot -> row
    const float* w;          // [T, top_k] or null (all 1)
    void* out;               // [T, H]
    int64_t nv;              // vectors per row
    int64_t units;           // T * segs
    int top_k, rows, segs;
};

// A warp per (token, 32 vectors of the row): the loads of four slots are issued before the first
// multiply.
template <MoeType TY, int VE>
__global__ void __launch_bounds__(kMoeThreads)
moe_unpermute_kernel(const UnpermuteArgs a) {
    using P = MoePack<TY, VE>;
    using V = typename P::V;
    const int lane = threadIdx.x & 31;
    const int64_t u = (int64_t)blockIdx.x * (kMoeThreads / 32) + (threadIdx.x >> 5);
    grid_dependency_wait();
    grid_launch_dependents();
    if (u >= a.units) return;
    const int64_t t = u / a.segs;
    const int sg = (int)(u % a.segs);
    const int k = a.top_k;
    int32_t my_row = -1;
    float my_w = 1.0f;
    if (lane < k) {
        my_row = a.idx[t * k + lane];
        if (a.w != nullptr) my_w = a.w[t * k + lane];
        if (my_row >= a.rows) {
            atomicExch(&g_device_error, kErrBadSlot);
            my_row = -1;
        }
    }
    const int64_t c = (int64_t)sg * 32 + lane;
    const bool on = c < a.nv;
    float acc[VE];
#pragma unroll
    for (int q = 0; q < VE; ++q) acc[q] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += 4) {
        V v[4];
        int32_t r[4];
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {                       // lanes past top_k hold row -1 (j0 + j < 32)
            r[j] = __shfl_sync(0xFFFFFFFFu, my_row, j0 + j);
            w[j] = __shfl_sync(0xFFFFFFFFu, my_w, j0 + j);
            if (r[j] >= 0 && on) v[j] = __ldg(reinterpret_cast<const V*>(a.y) + (int64_t)r[j] * a.nv + c);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (r[j] >= 0 && on) {
                float f[VE];
                P::unpack(v[j], f);
#pragma unroll
                for (int q = 0; q < VE; ++q) acc[q] = a.w != nullptr ? fmaf(w[j], f[q], acc[q]) : acc[q] + f[q];
            }
        }
    }
    if (on) reinterpret_cast<V*>(a.out)[t * a.nv + c] = P::pack(acc);
}

struct UnpermuteBwdArgs {
    const void* g;           // [T, H]
    const void* y;           // [rows, H] or null (no weights)
    const int32_t* idx;      // [T, top_k]
    const int32_t* inv;      // [rows]: row -> slot, -1 for padding
    const int32_t* total;    // m_indptr + E: the rows in use
    const float* w;          // [T, top_k] or null
    void* gy;                // [rows, H]
    float* gw;               // [T, top_k] or null
    int64_t nv;
    int T, top_k, rows;
};

// A CTA per token: g[t] is read once per four slots (from L1 after the first), each slot's row of y
// once; gy's rows are written and the four dot products kept per thread, then summed over the CTA
// in a fixed order.  The CTAs past T write zeros into the padding rows of the segments.
template <MoeType TY, int VE>
__global__ void __launch_bounds__(kMoeThreads)
moe_unpermute_bwd_kernel(const UnpermuteBwdArgs a) {
    using P = MoePack<TY, VE>;
    using V = typename P::V;
    __shared__ float part[4][kMoeThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    if (blockIdx.x >= a.T) {
        const int used = min(*a.total, a.rows);
        const int64_t step = (int64_t)(gridDim.x - a.T) * nw * 32;
        for (int64_t r0 = ((int64_t)(blockIdx.x - a.T) * nw + warp) * 32; r0 < used; r0 += step) {
            const bool pad = r0 + lane < used && a.inv[r0 + lane] < 0;
            uint32_t m = __ballot_sync(0xFFFFFFFFu, pad);
            while (m) {
                const int64_t r = r0 + __ffs(m) - 1;
                m &= m - 1;
                V* dst = reinterpret_cast<V*>(a.gy) + r * a.nv;
                for (int64_t q = lane; q < a.nv; q += 32) dst[q] = V{};
            }
        }
        return;
    }
    const int64_t t = blockIdx.x;
    const int k = a.top_k;
    const V* g = reinterpret_cast<const V*>(a.g) + t * a.nv;
    for (int j0 = 0; j0 < k; j0 += 4) {
        int32_t r[4];
        float w[4], dot[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[j] = j0 + j < k ? a.idx[t * k + j0 + j] : -1;
            w[j] = j0 + j < k && a.w != nullptr ? a.w[t * k + j0 + j] : 1.0f;
            if (r[j] >= a.rows) {
                if (tid == 0) atomicExch(&g_device_error, kErrBadSlot);
                r[j] = -1;
            }
        }
        for (int64_t c = tid; c < a.nv; c += blockDim.x) {
            const V gv = g[c];
            V yv[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (r[j] >= 0 && a.gw != nullptr) yv[j] = __ldg(reinterpret_cast<const V*>(a.y) + (int64_t)r[j] * a.nv + c);
            float gf[VE];
            P::unpack(gv, gf);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (r[j] < 0) continue;
                float o[VE];
                if (a.gw != nullptr) {
                    float yf[VE];
                    P::unpack(yv[j], yf);
#pragma unroll
                    for (int q = 0; q < VE; ++q) dot[j] = fmaf(gf[q], yf[q], dot[j]);
                }
#pragma unroll
                for (int q = 0; q < VE; ++q) o[q] = w[j] * gf[q];
                reinterpret_cast<V*>(a.gy)[(int64_t)r[j] * a.nv + c] = P::pack(o);
            }
        }
        if (a.gw != nullptr) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], d);
                if (lane == 0) part[j][warp] = dot[j];
            }
            __syncthreads();
            if (tid < 4 && j0 + tid < k) {
                float s = part[tid][0];
                for (int q = 1; q < nw; ++q) s += part[tid][q];
                a.gw[t * k + j0 + tid] = s;                 // an inactive slot's sums are all 0
            }
            __syncthreads();
        }
    }
}

}  // namespace nvfp4lora
