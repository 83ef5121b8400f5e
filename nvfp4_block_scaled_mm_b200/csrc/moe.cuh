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
//
// All of it is bound by HBM where there are many tokens (8 KB rows, 8 slots): sorting 8192 tokens 121 us
// (5.4 TB/s; about 10 us of it are the two launches and the counting), its gradient 89 us (6.4 TB/s), the weighted sum
// of 4096 tokens 47 us (6.1 TB/s) and its gradients 109 us (5.3 TB/s, half of it scattered writes).  A decode batch
// takes 6 us (64 tokens, 768 rows written, 645 of them padding) and 1.7 us, launch latency.  Rows off 16 bytes move one
// element per access: the weighted sum of 2056 x 10 rows of 3693 bf16 78 us (31 at 3696), its gradients 105 (68).
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
constexpr int kMoeBatchSlots = 64;       // slots ranked at a time by one CTA (kMoeMaxTopK at least)
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
moe_count_kernel(const int32_t* ids, int64_t n, int64_t chunk, int E, int32_t* counts) {
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
    // the first kMoeThreads threads hold PER experts each; further warps hold none
    __shared__ int32_t warp_seg[32], warp_pad[32];
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
    __syncthreads();
}

// One launch where every CTA can count all slots itself, two above kMoeSelfCountSlots (4096 slots 4.5 us; 16384
// slots 17 us in one launch and 9 in two).
// CTA c owns the tokens [T c / grid, T (c + 1) / grid).  It counts the slots of every expert before
// its own and in all (from the slots, or from the counting kernel's table plus the part of its own
// chunk), ranks its slots in order, and copies each of its tokens' rows to the token's up to top_k
// places, read once: a warp of its own ranks the next batch while the others copy.  Padding rows and the row -> slot table's -1 entries are shared out evenly.
constexpr int kMoePermuteThreads = kMoeThreads + 32;

template <int VB>
__global__ void __launch_bounds__(kMoePermuteThreads)
moe_permute_kernel(const PermuteArgs a) {
    using V = typename MoeVec<VB>::type;
    // vectors per lane and unit of copying: 8 of 16 bytes (121 us against 125 with 4 at 8192 tokens x 8 slots x 8 KB)
    constexpr int UN = VB == 16 ? 8 : 4;
    __shared__ int32_t before[kMoeMaxExperts];              // slots of the expert before the next one ranked
    __shared__ int32_t total[kMoeMaxExperts];
    __shared__ int32_t offs[kMoeMaxExperts + 1];
    __shared__ int32_t pads[kMoeMaxExperts + 1];
    __shared__ int32_t place[2][kMoeBatchSlots];
    constexpr int NT = kMoePermuteThreads, CW = kMoeThreads / 32;   // threads; copying warps
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = a.E, k = a.top_k;
    for (int e = tid; e < E; e += NT) { before[e] = 0; total[e] = 0; }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();

    const int t0 = (int)((int64_t)a.T * blockIdx.x / gridDim.x);
    const int t1 = (int)((int64_t)a.T * (blockIdx.x + 1) / gridDim.x);
    const int64_t start = (int64_t)t0 * k;
    if (a.counts == nullptr) {
        // total[] holds the slots from `start` on until the two are added below
        for (int64_t i0 = 0; i0 < a.n; i0 += 4 * NT) {
            int e[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t i = i0 + q * NT + tid;
                e[q] = i < a.n ? a.ids[i] : -1;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (e[q] >= 0 && e[q] < E) atomicAdd(i0 + q * NT + tid < start ? &before[e[q]] : &total[e[q]], 1);
                else if (e[q] >= E && blockIdx.x == 0) report_bad_entry(kErrBadSlot);
            }
        }
        __syncthreads();
        for (int e = tid; e < E; e += NT) total[e] += before[e];
    } else {
        const int own = (int)(start / a.chunk);             // chunks before this one lie before `start`
        for (int e = tid; e < E; e += NT) {
            int32_t b = 0, all = 0;
#pragma unroll 16
            for (int c = 0; c < kMoeCountChunks; ++c) {
                const int32_t v = a.counts[(int64_t)c * E + e];
                all += v;
                if (c < own) b += v;
            }
            before[e] = b;
            total[e] = all;
        }
        __syncthreads();
        for (int64_t i = own * a.chunk + tid; i < start; i += NT) {
            const int e = a.ids[i];
            if (e >= 0 && e < E) atomicAdd(&before[e], 1);
        }
    }
    __syncthreads();
    moe_scan(total, E, a.align, offs, pads);
    if (blockIdx.x == 0)
        for (int e = tid; e <= E; e += NT) a.indptr[e] = offs[e];

    // ---- this CTA's tokens, some at a time: rank their slots, copy their rows ----
    const int64_t nv = a.row_bytes / VB;
    const int segs = (int)((nv + 32 * UN - 1) / (32 * UN));
    const int batch = kMoeBatchSlots / k;
    auto rank = [&](int tb, int32_t* dst) {
        const int ns = min(batch, t1 - tb) * k;
        for (int s = 0; s < ns; s += 32) {
            const int64_t i = (int64_t)tb * k + s + lane;
            const bool in = s + lane < ns;
            int e = in ? a.ids[i] : -1;
            if (e >= E) {
                if (a.counts != nullptr) report_bad_entry(kErrBadSlot);
                e = -1;
            }
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
            int32_t row = -1;
            if (e >= 0) row = offs[e] + before[e] + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (e >= 0 && lane == __ffs(same) - 1) before[e] += __popc(same);
            __syncwarp();
            if (in) {
                dst[s + lane] = row;
                a.idx[i] = row;
                if (row >= 0) a.inv[row] = (int32_t)i;
            }
        }
    };
    if (warp == CW && t0 < t1) rank(t0, place[0]);
    __syncthreads();
    for (int tb = t0, cur = 0; tb < t1; tb += batch, cur ^= 1) {
        if (warp == CW) {
            if (tb + batch < t1) rank(tb + batch, place[cur ^ 1]);
        } else {
            const int nt = min(batch, t1 - tb);
            for (int u = warp; u < nt * segs; u += CW) {
                const int t = u / segs, sg = u % segs;
                const V* src = reinterpret_cast<const V*>(a.x + (int64_t)(tb + t) * a.row_bytes) + (int64_t)sg * 32 * UN;
                const int64_t left = nv - (int64_t)sg * 32 * UN;
                V v[UN];
#pragma unroll
                for (int q = 0; q < UN; ++q)
                    if (q * 32 + lane < left) v[q] = src[q * 32 + lane];
                for (int j = 0; j < k; ++j) {
                    const int32_t row = place[cur][t * k + j];
                    if (row < 0) continue;
                    V* dst = reinterpret_cast<V*>(a.rows + (int64_t)row * a.row_bytes) + (int64_t)sg * 32 * UN;
#pragma unroll
                    for (int q = 0; q < UN; ++q)
                        if (q * 32 + lane < left) dst[q * 32 + lane] = v[q];
                }
            }
        }
        __syncthreads();
    }

    // ---- padding rows, and the -1 entries of the row -> slot table ----
    const int npad = pads[E];
    const int gw = blockIdx.x * (NT / 32) + warp, nw = gridDim.x * (NT / 32);
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
    for (int64_t r = (int64_t)offs[E] + blockIdx.x * NT + tid; r < a.capacity; r += gridDim.x * NT)
        a.inv[r] = -1;
}

// ---------------------------------------------------------------------------------------
// back: the weighted sum of a token's rows
// ---------------------------------------------------------------------------------------

enum class MoeType { BF16, FP16, FP32 };

template <MoeType TY> struct MoeElem { using type = uint16_t; };
template <> struct MoeElem<MoeType::FP32> { using type = float; };

template <MoeType TY>
__device__ __forceinline__ float to_f32(typename MoeElem<TY>::type h) {
    if constexpr (TY == MoeType::FP32) return h;
    else if constexpr (TY == MoeType::BF16) return __uint_as_float((uint32_t)h << 16);
    else return __half2float(__ushort_as_half(h));
}

template <MoeType TY>
__device__ __forceinline__ typename MoeElem<TY>::type from_f32(float f) {   // nearest, ties to even
    if constexpr (TY == MoeType::FP32) return f;
    else if constexpr (TY == MoeType::BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(f));
    else return __half_as_ushort(__float2half_rn(f));
}

// A warp's share of a row: 256 elements from element e0 on, eight per lane.  VEC: the lane's eight are
// neighbours, one 16-byte access (two for fp32, each bounded by itself: a row of 12 ends between a lane's two);
// rows are whole numbers of 16 bytes long and start on 16-byte boundaries.  EIGHT: the length is a multiple of 8, and
// one bound serves a lane (the norm of 4096 x 12288 fp32, where the second one spills: 115 us, 123 with it).  Without
// VEC they are 32 apart, so that any alignment is read and written in coalesced element accesses.
template <MoeType TY, bool VEC, bool EIGHT = false>
struct RowChunk {
    using E = typename MoeElem<TY>::type;
    static constexpr int NW = 8 * (int)sizeof(E) / 16;
    static constexpr int PER = 16 / (int)sizeof(E);        // elements of a 16-byte access
    union Raw {
        uint4 w[NW];
        E e[8];
    };
    static __device__ __forceinline__ int64_t at(int64_t e0, int lane, int i) {
        return VEC ? e0 + lane * 8 + i : e0 + i * 32 + lane;
    }
    static __device__ __forceinline__ Raw load(const void* row, int64_t e0, int64_t H, int lane) {
        Raw r;
        const E* p = static_cast<const E*>(row);
        if constexpr (VEC && EIGHT) {
            if (at(e0, lane, 0) < H) {
#pragma unroll
                for (int i = 0; i < NW; ++i) r.w[i] = reinterpret_cast<const uint4*>(p + at(e0, lane, 0))[i];
            } else {
#pragma unroll
                for (int i = 0; i < NW; ++i) r.w[i] = make_uint4(0, 0, 0, 0);
            }
        } else if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < NW; ++i)
                r.w[i] = at(e0, lane, i * PER) < H ? reinterpret_cast<const uint4*>(p + at(e0, lane, 0))[i] : make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) r.e[i] = at(e0, lane, i) < H ? p[at(e0, lane, i)] : E(0);
        }
        return r;
    }
    static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[8]) {
        if constexpr (TY == MoeType::FP32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = r.e[i];
        } else {
            const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = to_f32<TY>((uint16_t)(u[i] & 0xFFFFu));
                f[2 * i + 1] = to_f32<TY>((uint16_t)(u[i] >> 16));
            }
        }
    }
    static __device__ __forceinline__ void store(void* row, int64_t e0, int64_t H, int lane, const float (&f)[8]) {
        E* p = static_cast<E*>(row);
        Raw r;
        if constexpr (TY == MoeType::FP32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) r.e[i] = f[i];
        } else {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[i] = (uint32_t)from_f32<TY>(f[2 * i]) | ((uint32_t)from_f32<TY>(f[2 * i + 1]) << 16);
            r.w[0] = make_uint4(u[0], u[1], u[2], u[3]);
        }
        if constexpr (VEC && EIGHT) {
            if (at(e0, lane, 0) < H) {
#pragma unroll
                for (int i = 0; i < NW; ++i) reinterpret_cast<uint4*>(p + at(e0, lane, 0))[i] = r.w[i];
            }
        } else if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < NW; ++i)
                if (at(e0, lane, i * PER) < H) reinterpret_cast<uint4*>(p + at(e0, lane, 0))[i] = r.w[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (at(e0, lane, i) < H) p[at(e0, lane, i)] = r.e[i];
        }
    }
};

struct UnpermuteArgs {
    const void* y;           // [rows, H]
    const int32_t* idx;      // [T, top_k]: slot -> row
    const float* w;          // [T, top_k] or null (all 1)
    void* out;               // [T, H]
    int64_t H;
    int64_t units;           // T * segs
    int top_k, rows, segs;   // segs = ceil(H / 256)
};

template <MoeType TY>
__device__ __forceinline__ const void* row_at(const void* base, int64_t row, int64_t H) {
    return static_cast<const typename MoeElem<TY>::type*>(base) + row * H;
}

template <MoeType TY>
__device__ __forceinline__ void* row_at(void* base, int64_t row, int64_t H) {
    return static_cast<typename MoeElem<TY>::type*>(base) + row * H;
}

// A warp per (token, 256 elements of the row): the loads of four slots (two of fp32) are issued before the
// first multiply.
template <MoeType TY, bool VEC>
__global__ void __launch_bounds__(kMoeThreads)
moe_unpermute_kernel(const UnpermuteArgs a) {
    using C = RowChunk<TY, VEC>;
    constexpr int JC = TY == MoeType::FP32 ? 2 : 4;
    const int lane = threadIdx.x & 31;
    const int64_t u = (int64_t)blockIdx.x * (kMoeThreads / 32) + (threadIdx.x >> 5);
    grid_dependency_wait();
    grid_launch_dependents();
    if (u >= a.units) return;
    const int64_t t = u / a.segs, e0 = (u - t * a.segs) * 256;
    const int k = a.top_k;
    int32_t my_row = -1;
    float my_w = 1.0f;
    if (lane < k) {
        my_row = a.idx[t * k + lane];
        if (a.w != nullptr) my_w = a.w[t * k + lane];
        if (my_row >= a.rows) {
            report_bad_entry(kErrBadSlot);
            my_row = -1;
        }
    }
    float acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += JC) {
        typename C::Raw v[JC];
        int32_t r[JC];
        float w[JC];
#pragma unroll
        for (int j = 0; j < JC; ++j) {                      // lanes past top_k hold row -1 (j0 + j < 32)
            r[j] = __shfl_sync(0xFFFFFFFFu, my_row, j0 + j);
            w[j] = __shfl_sync(0xFFFFFFFFu, my_w, j0 + j);
            if (r[j] >= 0) v[j] = C::load(row_at<TY>(a.y, r[j], a.H), e0, a.H, lane);
        }
#pragma unroll
        for (int j = 0; j < JC; ++j) {
            if (r[j] >= 0) {
                float f[8];
                C::unpack(v[j], f);
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[q] = a.w != nullptr ? fmaf(w[j], f[q], acc[q]) : acc[q] + f[q];
            }
        }
    }
    C::store(row_at<TY>(a.out, t, a.H), e0, a.H, lane, acc);
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
    int64_t H;
    int T, top_k, rows;
};

// A CTA per token: g[t] is read once per two slots (from L1 after the first), each slot's row of y once; gy's
// rows are written and the two dot products kept per thread, then summed over the CTA in a fixed order.  The
// CTAs past T write zeros into the padding rows of the segments.  128 threads and two slots at a time: 109 us at
// 4096 tokens x 8 slots x 8 KB (5.3 TB/s); 256 threads and four slots 114, eight slots 128 (fewer CTAs resident).
constexpr int kMoeBwdThreads = 128;
constexpr int kMoeBwdSlots = 2;

template <MoeType TY, bool VEC>
__global__ void __launch_bounds__(kMoeBwdThreads)
moe_unpermute_bwd_kernel(const UnpermuteBwdArgs a) {
    using C = RowChunk<TY, VEC>;
    constexpr int JC = kMoeBwdSlots;
    __shared__ float part[JC][kMoeBwdThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    if (blockIdx.x >= a.T) {
        const int used = min(*a.total, a.rows);
        const int64_t step = (int64_t)(gridDim.x - a.T) * nw * 32;
        const float zero[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        for (int64_t r0 = ((int64_t)(blockIdx.x - a.T) * nw + warp) * 32; r0 < used; r0 += step) {
            const bool pad = r0 + lane < used && a.inv[r0 + lane] < 0;
            uint32_t m = __ballot_sync(0xFFFFFFFFu, pad);
            while (m) {
                void* row = row_at<TY>(a.gy, r0 + __ffs(m) - 1, a.H);
                m &= m - 1;
                for (int64_t e0 = 0; e0 < a.H; e0 += 256) C::store(row, e0, a.H, lane, zero);
            }
        }
        return;
    }
    const int64_t t = blockIdx.x;
    const int k = a.top_k;
    const void* g = row_at<TY>(a.g, t, a.H);
    for (int j0 = 0; j0 < k; j0 += JC) {
        int32_t r[JC];
        float w[JC], dot[JC];
#pragma unroll
        for (int j = 0; j < JC; ++j) {
            dot[j] = 0.0f;
            r[j] = j0 + j < k ? a.idx[t * k + j0 + j] : -1;
            w[j] = j0 + j < k && a.w != nullptr ? a.w[t * k + j0 + j] : 1.0f;
            if (r[j] >= a.rows) {
                if (tid == 0) report_bad_entry(kErrBadSlot);
                r[j] = -1;
            }
        }
        for (int64_t e0 = (int64_t)warp * 256; e0 < a.H; e0 += nw * 256) {
            const typename C::Raw gv = C::load(g, e0, a.H, lane);
            typename C::Raw yv[JC];
#pragma unroll
            for (int j = 0; j < JC; ++j)
                if (r[j] >= 0 && a.gw != nullptr) yv[j] = C::load(row_at<TY>(a.y, r[j], a.H), e0, a.H, lane);
            float gf[8];
            C::unpack(gv, gf);
#pragma unroll
            for (int j = 0; j < JC; ++j) {
                if (r[j] < 0) continue;
                float o[8];
                if (a.gw != nullptr) {
                    float yf[8];
                    C::unpack(yv[j], yf);
#pragma unroll
                    for (int q = 0; q < 8; ++q) dot[j] = fmaf(gf[q], yf[q], dot[j]);
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) o[q] = w[j] * gf[q];
                C::store(row_at<TY>(a.gy, r[j], a.H), e0, a.H, lane, o);
            }
        }
        if (a.gw != nullptr) {
#pragma unroll
            for (int j = 0; j < JC; ++j) {
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], d);
                if (lane == 0) part[j][warp] = dot[j];
            }
            __syncthreads();
            if (tid < JC && j0 + tid < k) {
                float s = part[tid][0];
                for (int q = 1; q < nw; ++q) s += part[tid][q];
                a.gw[t * k + j0 + tid] = s;                 // an inactive slot's sums are all 0
            }
            __syncthreads();
        }
    }
}

}  // namespace nvfp4lora
