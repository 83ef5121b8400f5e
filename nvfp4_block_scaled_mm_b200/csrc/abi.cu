// C ABI of the NVFP4 + LoRA GEMM library (declared in include/nvfp4lora.h).
//
// Host side: argument rules (flashinfer.gemm.mm_nvfp4_lora, Notes: Shape rules; Parameters),
// adapter pins and stale checks (Parameters: lora_adapter; Notes: CUDA graphs), the eager
// prepare's single host read and checks (prepare_nvfp4_lora_adapter, Parameters: alpha,
// Returns), TMA descriptor encoding, and kernel launch.  Every rule is checked before any
// CUDA call, so a rejected call enqueues nothing.  This is the library's only translation
// unit: it includes the kernels and the device error word they set.

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <atomic>
#include <initializer_list>
#include <mutex>
#include <set>
#include <string>
#include <type_traits>

#include "../../include/nvfp4lora.h"
#include "bgmv.cuh"
#include "fold.cuh"
#include "fp8_gemm.cuh"
#include "fp8_quant.cuh"
#include "fp8_splitk.cuh"
#include "gemm.cuh"
#include "gemm_decode.cuh"
#include "gemm_pair.cuh"
#include "moe.cuh"
#include "ptx.cuh"
#include "quantize.cuh"
#include "selftest.cuh"

namespace nvfp4lora {
namespace {

thread_local std::string t_last_error;

nvfp4lora_status fail(nvfp4lora_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    t_last_error = buf;
    return st;
}

nvfp4lora_status cuda_fail(cudaError_t e, const char* what) {
    return fail(NVFP4LORA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// ---------------------------------------------------------------------------------------
// device facts, cached per device
// ---------------------------------------------------------------------------------------

constexpr int kMaxDevices = 64;

struct DeviceInfo {
    bool init = false;
    bool supported = false;
    int sms = 0;
    int major = 0, minor = 0;
    std::set<const void*> smem_attr_set;   // kernels whose dynamic shared memory limit is raised
};

std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];

nvfp4lora_status device_info(int* dev_out, DeviceInfo** info_out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(NVFP4LORA_ERR_CUDA, "device ordinal %d out of range", dev);
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceInfo& d = g_dev[dev];
    if (!d.init) {
        if ((e = cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&d.minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
            return cuda_fail(e, "cudaDeviceGetAttribute");
        d.supported = (d.major == 10 && d.minor == 0);
        d.init = true;
    }
    if (!d.supported)
        return fail(NVFP4LORA_ERR_UNSUPPORTED_ARCH,
                    "device %d is sm_%d%d; this library runs on sm_100 (B200) only", dev, d.major, d.minor);
    *dev_out = dev;
    *info_out = &d;
    return NVFP4LORA_OK;
}

template <typename Kernel>
nvfp4lora_status ensure_smem_attr(DeviceInfo* info, Kernel kernel, int smem, bool max_carveout = true) {
    std::lock_guard<std::mutex> lock(g_mu);
    const void* key = reinterpret_cast<const void*>(kernel);
    if (info->smem_attr_set.count(key)) return NVFP4LORA_OK;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    // the whole unified L1 / shared array as shared memory, so co-resident CTAs fit
    if (e == cudaSuccess && max_carveout)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    info->smem_attr_set.insert(key);
    return NVFP4LORA_OK;
}

// ---------------------------------------------------------------------------------------
// TMA descriptors
// ---------------------------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;
cudaError_t g_encode_err = cudaSuccess;

nvfp4lora_status get_encoder(PFN_cuTensorMapEncodeTiled_v12000* out) {
    std::call_once(g_encode_once, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        g_encode_err = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q);
        if (g_encode_err == cudaSuccess && q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    if (g_encode == nullptr)
        return fail(NVFP4LORA_ERR_CUDA, "cuTensorMapEncodeTiled unavailable (%s)",
                    cudaGetErrorString(g_encode_err));
    *out = g_encode;
    return NVFP4LORA_OK;
}

// 2-D row-major tensor [rows, cols] of `esize`-byte elements, read in boxes of
// box_cols x box_rows with the 128-byte swizzle; out-of-range elements read as zero.
// The LoRA operands d [M, r] and lora_b / b_folded [N, r] of the tiled kernels are read with no L2
// promotion.  Their boxes are 64 columns wide and zero-filled past r; where r is not a multiple of
// 16 a row's in-bounds part ends inside a 32-byte sector, and with 256-byte promotion those loads
// arrived late enough to stall the tile's end: raw path, M = 256, N = 14336, K = 4096, r = 8 ran
// 18.3 us on the SM-pair kernel with promotion and 16.9 without (r = 16: 14.9 either way).
constexpr CUtensorMapL2promotion kLoraPromotion = CU_TENSOR_MAP_L2_PROMOTION_NONE;

nvfp4lora_status encode_2d(CUtensorMap* map, const void* base, CUtensorMapDataType dtype, int esize,
                           uint64_t cols, uint64_t rows, uint32_t box_cols, uint32_t box_rows,
                           CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B,
                           CUtensorMapL2promotion promotion = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    nvfp4lora_status st = get_encoder(&enc);
    if (st != NVFP4LORA_OK) return st;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols * (uint64_t)esize};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, dtype, 2, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(NVFP4LORA_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
    return NVFP4LORA_OK;
}

// 3-D view of a row-major [rows, cols] uint8 matrix as (128-byte chunk, row, chunk index), used
// to name one 128-row block across several K chunks in a single box (L2 prefetch only).
nvfp4lora_status encode_rows_by_chunks(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows,
                                       uint32_t box_rows, uint32_t box_chunks) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    nvfp4lora_status st = get_encoder(&enc);
    if (st != NVFP4LORA_OK) return st;
    cuuint64_t dims[3] = {128, rows, cols / 128};
    cuuint64_t strides[2] = {cols, 128};
    cuuint32_t box[3] = {128, box_rows, box_chunks};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(NVFP4LORA_ERR_CUDA, "cuTensorMapEncodeTiled (3-D) failed (CUresult %d)", (int)r);
    return NVFP4LORA_OK;
}

// ---------------------------------------------------------------------------------------
// argument rules
// ---------------------------------------------------------------------------------------

constexpr int64_t kMaxDim = (int64_t)1 << 30;   // keeps every tile coordinate in int32
constexpr int64_t kMaxK = (int64_t)1 << 20;

nvfp4lora_status check_rank(int64_t r) {
    if (r < 8 || r > 128 || r % 8 != 0)
        return fail(NVFP4LORA_ERR_INVALID_ARG,
                    "LoRA rank r = %lld: r must be a multiple of 8 in [8, 128]", (long long)r);
    return NVFP4LORA_OK;
}

nvfp4lora_status check_base(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, int64_t a_sf_bytes,
                            const uint8_t* b_sf, int64_t b_sf_bytes, const float* alpha,
                            const uint16_t* bias, const uint16_t* out, int64_t M, int64_t N, int64_t K) {
    if (M < 1) return fail(NVFP4LORA_ERR_INVALID_ARG, "M = %lld: M >= 1 is required", (long long)M);
    if (N < 1) return fail(NVFP4LORA_ERR_INVALID_ARG, "N = %lld: N >= 1 is required", (long long)N);
    if (K < 256 || K % 256 != 0)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "K = %lld: K must be a positive multiple of 256", (long long)K);
    if (M > kMaxDim || N > kMaxDim || K > kMaxK)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "M, N <= 2^30 and K <= 2^20 are required");
    if (!a || !b || !a_sf || !b_sf || !alpha || !out)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "a, b, a_sf, b_sf, alpha and out must be non-null");
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_sf, 16) || !aligned(b_sf, 16) || !aligned(out, 16))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "a, b, a_sf, b_sf and out must be 16-byte aligned");
    if (!aligned(alpha, 4)) return fail(NVFP4LORA_ERR_INVALID_ARG, "alpha must be 4-byte aligned");
    if (bias && !aligned(bias, 2)) return fail(NVFP4LORA_ERR_INVALID_ARG, "bias must be 2-byte aligned");
    const int64_t need_a = (M + 127) / 128 * 128 * (K / 16);
    const int64_t need_b = (N + 127) / 128 * 128 * (K / 16);
    if (a_sf_bytes < need_a)
        return fail(NVFP4LORA_ERR_INVALID_ARG,
                    "a_sf has %lld bytes; the 128x4 layout with rows padded to 128 needs %lld",
                    (long long)a_sf_bytes, (long long)need_a);
    if (b_sf_bytes < need_b)
        return fail(NVFP4LORA_ERR_INVALID_ARG,
                    "b_sf has %lld bytes; the 128x4 layout with rows padded to 128 needs %lld",
                    (long long)b_sf_bytes, (long long)need_b);
    return NVFP4LORA_OK;
}

// ---------------------------------------------------------------------------------------
// GEMM launch
// ---------------------------------------------------------------------------------------

constexpr int kStages = 3;

// The tiled kernels split their registers by warpgroup (setmaxnreg); the split assumes the per-
// thread count the compiler gave the kernel at launch.  A smaller count would leave the epilogue
// warpgroups waiting for registers that never come, so a build that differs is refused here.
template <typename Kernel>
nvfp4lora_status check_split_regs(Kernel kernel, int expected, std::atomic<int>& checked, const char* what) {
    if (checked.load(std::memory_order_relaxed)) return NVFP4LORA_OK;
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return cuda_fail(e, what);
    if (fa.numRegs != expected)
        return fail(NVFP4LORA_ERR_CUDA, "%s built with %d registers per thread, its register split assumes %d", what,
                    fa.numRegs, expected);
    checked.store(1, std::memory_order_relaxed);
    return NVFP4LORA_OK;
}

template <Mode MODE>
nvfp4lora_status launch_gemm(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, const uint8_t* b_sf,
                             const float* alpha, const float* scale, const uint16_t* d,
                             const uint16_t* lb, int64_t r, const uint16_t* bias, uint16_t* out,
                             int64_t M, int64_t N, int64_t K, cudaStream_t stream) {
    int dev = 0;
    DeviceInfo* info = nullptr;
    nvfp4lora_status st = device_info(&dev, &info);
    if (st != NVFP4LORA_OK) return st;

    auto kernel = nvfp4_gemm_kernel<kStages, MODE>;
    constexpr int smem = GemmSmem<kStages>::DYN_BYTES;
    if ((st = ensure_smem_attr(info, kernel, smem)) != NVFP4LORA_OK) return st;
    static std::atomic<int> regs_ok{0};            // one per instantiation
    if ((st = check_split_regs(kernel, kGemmRegsLaunch, regs_ok, "GEMM")) != NVFP4LORA_OK) return st;

    CUtensorMap tm_a, tm_b, tm_d, tm_lb, tm_out;
    std::memset(&tm_d, 0, sizeof(tm_d));
    std::memset(&tm_lb, 0, sizeof(tm_lb));
    std::memset(&tm_out, 0, sizeof(tm_out));
    if ((st = encode_2d(&tm_a, a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K / 2, M, 128, kTileM)) != NVFP4LORA_OK) return st;
    if ((st = encode_2d(&tm_b, b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K / 2, N, 128, kTileN)) != NVFP4LORA_OK) return st;
    if (MODE != Mode::Off) {
        if ((st = encode_2d(&tm_d, d, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, r, M, 64, kTileM, CU_TENSOR_MAP_SWIZZLE_128B, kLoraPromotion)) != NVFP4LORA_OK) return st;
        if ((st = encode_2d(&tm_lb, lb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, r, N, 64, kTileN, CU_TENSOR_MAP_SWIZZLE_128B, kLoraPromotion)) != NVFP4LORA_OK) return st;
    }
    // rows of out 16-byte aligned: the epilogue writes 32 x 32 bf16 boxes with TMA stores
    const bool vec_out = (N % 8 == 0 && (bias == nullptr || aligned(bias, 16)));
    if (vec_out &&
        (st = encode_2d(&tm_out, out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, N, M, kOutBoxCols, kOutBoxRows,
                        CU_TENSOR_MAP_SWIZZLE_NONE)) != NVFP4LORA_OK)
        return st;

    GemmArgs args;
    args.a_sf = a_sf;
    args.b_sf = b_sf;
    args.alpha = alpha;
    args.scale = scale;
    args.bias = bias;
    args.out = out;
    args.M = (int)M;
    args.N = (int)N;
    args.K = (int)K;
    args.r = (int)r;
    args.m_tiles = (int)((M + kTileM - 1) / kTileM);
    args.n_tiles = (int)((N + kTileN - 1) / kTileN);
    const int64_t tiles = (int64_t)args.m_tiles * args.n_tiles;
    if (tiles > INT32_MAX) return fail(NVFP4LORA_ERR_INVALID_ARG, "too many output tiles (M x N too large)");
    args.num_tiles = (int)tiles;
    args.k_stages = (int)(K / 256);
    args.sf_atoms_k = (int)(K / 64);
    args.sf_row_blocks_b = (int)((N + 127) / 128);
    args.vec_out = vec_out ? 1 : 0;
    args.m_indptr = nullptr;
    args.num_experts = 0;

    const int grid = (int)std::min<int64_t>(tiles, info->sms);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tm_a, tm_b, tm_d, tm_lb, tm_out, args);
    if (e != cudaSuccess) return cuda_fail(e, "GEMM launch");
    return NVFP4LORA_OK;
}

// Grouped call (nvfp4lora_grouped_mm): the single-SM tiled kernel over 128-row blocks whose expert
// comes from m_indptr on the device.  `rows` is the row count of a, d and out; b and lora_b are
// [E * N, .] row-major; alpha is [E].
template <Mode MODE>
nvfp4lora_status launch_gemm_grouped(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, const uint8_t* b_sf,
                                     const int* m_indptr, int64_t E, const float* alpha, const float* scale,
                                     const uint16_t* d, const uint16_t* lb, int64_t r, const uint16_t* bias,
                                     uint16_t* out, int64_t rows, int64_t N, int64_t K, cudaStream_t stream) {
    int dev = 0;
    DeviceInfo* info = nullptr;
    nvfp4lora_status st = device_info(&dev, &info);
    if (st != NVFP4LORA_OK) return st;

    auto kernel = nvfp4_gemm_kernel<kStages, MODE, true>;
    constexpr int smem = GemmSmem<kStages>::DYN_BYTES;
    if ((st = ensure_smem_attr(info, kernel, smem)) != NVFP4LORA_OK) return st;
    static std::atomic<int> regs_ok{0};            // one per instantiation
    if ((st = check_split_regs(kernel, kGemmRegsLaunch, regs_ok, "grouped GEMM")) != NVFP4LORA_OK) return st;

    CUtensorMap tm_a, tm_b, tm_d, tm_lb, tm_out;
    std::memset(&tm_d, 0, sizeof(tm_d));
    std::memset(&tm_lb, 0, sizeof(tm_lb));
    std::memset(&tm_out, 0, sizeof(tm_out));
    if ((st = encode_2d(&tm_a, a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K / 2, rows, 128, kTileM)) != NVFP4LORA_OK) return st;
    if ((st = encode_2d(&tm_b, b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K / 2, E * N, 128, kTileN)) != NVFP4LORA_OK) return st;
    if (MODE != Mode::Off) {
        if ((st = encode_2d(&tm_d, d, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, r, rows, 64, kTileM, CU_TENSOR_MAP_SWIZZLE_128B, kLoraPromotion)) != NVFP4LORA_OK) return st;
        if ((st = encode_2d(&tm_lb, lb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, r, E * N, 64, kTileN, CU_TENSOR_MAP_SWIZZLE_128B, kLoraPromotion)) != NVFP4LORA_OK) return st;
    }
    const bool vec_out = (N % 8 == 0 && (bias == nullptr || aligned(bias, 16)));
    if (vec_out &&
        (st = encode_2d(&tm_out, out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, N, rows, kOutBoxCols, kOutBoxRows,
                        CU_TENSOR_MAP_SWIZZLE_NONE)) != NVFP4LORA_OK)
        return st;

    GemmArgs args;
    args.a_sf = a_sf;
    args.b_sf = b_sf;
    args.alpha = alpha;
    args.scale = scale;
    args.bias = bias;
    args.out = out;
    args.M = (int)rows;
    args.N = (int)N;
    args.K = (int)K;
    args.r = (int)r;
    args.m_tiles = (int)((rows + kTileM - 1) / kTileM);     // bound: the kernel reads m_indptr[E]
    args.n_tiles = (int)((N + kTileN - 1) / kTileN);
    const int64_t tiles = (int64_t)args.m_tiles * args.n_tiles;
    if (tiles > INT32_MAX) return fail(NVFP4LORA_ERR_INVALID_ARG, "too many output tiles (rows x N too large)");
    args.num_tiles = (int)tiles;
    args.k_stages = (int)(K / 256);
    args.sf_atoms_k = (int)(K / 64);
    args.sf_row_blocks_b = (int)((N + 127) / 128);         // per expert
    args.vec_out = vec_out ? 1 : 0;
    args.m_indptr = m_indptr;
    args.num_experts = (int)E;

    const int grid = (int)std::min<int64_t>(tiles, info->sms);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tm_a, tm_b, tm_d, tm_lb, tm_out, args);
    if (e != cudaSuccess) return cuda_fail(e, "grouped GEMM launch");
    return NVFP4LORA_OK;
}

// ---------------------------------------------------------------------------------------
// decode launch (M <= kDecodeMaxM): swapped operands, split-K over a cluster
// ---------------------------------------------------------------------------------------

constexpr int kDecodeMaxM = 32;

// Largest cluster split S <= max_s (a power of two) that keeps n_tiles * S CTAs within one wave
// and divides the K stages.
int decode_splits(int n_tiles, int k_stages, int sms, int max_s) {
    for (int s = max_s; s > 1; s >>= 1)
        if (k_stages % s == 0 && (int64_t)n_tiles * s <= sms) return s;
    return 1;
}

// STAGES ring slots (all of a split's K stages in flight where they fit); MAXS - 1 peer partial
// slots plus one for the LoRA accumulator on rank 0.
template <int MT, int STAGES, int MAXS, Mode MODE>
nvfp4lora_status launch_decode_plan(DeviceInfo* info, int splits, const uint8_t* a, const uint8_t* b,
                                    const uint8_t* a_sf, const uint8_t* b_sf, const float* alpha,
                                    const float* scale, const uint16_t* d, const uint16_t* lb, int64_t r,
                                    const uint16_t* bias, uint16_t* out, int64_t M, int64_t N, int64_t K,
                                    cudaStream_t stream) {
    nvfp4lora_status st;
    auto kernel = nvfp4_decode_kernel<MT, STAGES, MAXS, MODE>;
    constexpr int smem = DecodeSmem<MT, STAGES, MAXS>::DYN_BYTES;
    if ((st = ensure_smem_attr(info, kernel, smem)) != NVFP4LORA_OK) return st;

    CUtensorMap tm_a, tm_b, tm_d, tm_lb;
    std::memset(&tm_d, 0, sizeof(tm_d));
    std::memset(&tm_lb, 0, sizeof(tm_lb));
    if ((st = encode_2d(&tm_a, a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K / 2, M, 128, MT)) != NVFP4LORA_OK) return st;
    if ((st = encode_2d(&tm_b, b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K / 2, N, 128, 128)) != NVFP4LORA_OK) return st;
    if (MODE != Mode::Off) {
        if ((st = encode_2d(&tm_d, d, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, r, M, 64, MT)) != NVFP4LORA_OK) return st;
        if ((st = encode_2d(&tm_lb, lb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, r, N, 64, 128)) != NVFP4LORA_OK) return st;
    }
    DecodeArgs args;
    args.a_sf = a_sf;
    args.b_sf = b_sf;
    args.alpha = alpha;
    args.scale = scale;
    args.lb = lb;
    args.bias = bias;
    args.out = out;
    args.M = (int)M;
    args.N = (int)N;
    args.K = (int)K;
    args.r = (int)r;
    args.n_tiles = (int)((N + 127) / 128);
    const int k_stages = (int)(K / 256);
    args.splits = splits;
    args.stages_per_split = k_stages / args.splits;
    args.sf_atoms_k = (int)(K / 64);
    args.sf_row_blocks_b = (int)((N + 127) / 128);

    CUtensorMap tm_b3;
    // one prefetch box covers up to 8 chunks (128 KB, within the tensor-map box limit)
    args.pf_chunks = std::min(args.stages_per_split, 8);
    if ((st = encode_rows_by_chunks(&tm_b3, b, K / 2, N, 128, args.pf_chunks)) != NVFP4LORA_OK) return st;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(args.n_tiles, args.splits);
    cfg.blockDim = dim3(kDecodeThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (args.splits > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 1;
        attr[1].val.clusterDim.y = args.splits;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tm_a, tm_b, tm_d, tm_lb, tm_b3, args);
    if (e != cudaSuccess) return cuda_fail(e, "decode GEMM launch");
    return NVFP4LORA_OK;
}

// A split cluster (S > 1) streams few K stages per CTA: 4 slots hold them all at the workload
// shapes.  Without a split (many weight row blocks) one CTA streams the whole of K, and the ring is
// as deep as shared memory allows, since a CTA's streaming rate is its bytes in flight over the
// memory latency (M = 1, N = 14336, K = 4096: 10.0 us per call with 4 slots, 8.6 with 8).
template <int MT, Mode MODE>
nvfp4lora_status launch_decode_mt(DeviceInfo* info, const uint8_t* a, const uint8_t* b, const uint8_t* a_sf,
                                  const uint8_t* b_sf, const float* alpha, const float* scale, const uint16_t* d,
                                  const uint16_t* lb, int64_t r, const uint16_t* bias, uint16_t* out,
                                  int64_t M, int64_t N, int64_t K, cudaStream_t stream) {
    constexpr int MAXS = 4;
    constexpr int DEEP = (MT == 16) ? 8 : 6;
    const int n_tiles = (int)((N + 127) / 128);
    const int splits = decode_splits(n_tiles, (int)(K / 256), info->sms, MAXS);
    if (splits > 1)
        return launch_decode_plan<MT, 4, MAXS, MODE>(info, splits, a, b, a_sf, b_sf, alpha, scale, d, lb, r, bias,
                                                     out, M, N, K, stream);
    return launch_decode_plan<MT, DEEP, 1, MODE>(info, 1, a, b, a_sf, b_sf, alpha, scale, d, lb, r, bias, out, M,
                                                 N, K, stream);
}

template <Mode MODE>
nvfp4lora_status launch_decode(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, const uint8_t* b_sf,
                               const float* alpha, const float* scale, const uint16_t* d, const uint16_t* lb,
                               int64_t r, const uint16_t* bias, uint16_t* out, int64_t M, int64_t N, int64_t K,
                               cudaStream_t stream) {
    int dev = 0;
    DeviceInfo* info = nullptr;
    nvfp4lora_status st = device_info(&dev, &info);
    if (st != NVFP4LORA_OK) return st;
    if (M <= 16)
        return launch_decode_mt<16, MODE>(info, a, b, a_sf, b_sf, alpha, scale, d, lb, r, bias, out, M, N, K, stream);
    return launch_decode_mt<32, MODE>(info, a, b, a_sf, b_sf, alpha, scale, d, lb, r, bias, out, M, N, K, stream);
}

// ---------------------------------------------------------------------------------------
// SM-pair tiled launch: clusters of 2 CTAs, 256 x 256 tiles
// ---------------------------------------------------------------------------------------

template <Mode MODE>
nvfp4lora_status launch_gemm_pair(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, const uint8_t* b_sf,
                                  const float* alpha, const float* scale, const uint16_t* d, const uint16_t* lb,
                                  int64_t r, const uint16_t* bias, uint16_t* out, int64_t M, int64_t N, int64_t K,
                                  cudaStream_t stream) {
    int dev = 0;
    DeviceInfo* info = nullptr;
    nvfp4lora_status st = device_info(&dev, &info);
    if (st != NVFP4LORA_OK) return st;
    auto kernel = nvfp4_gemm_pair_kernel<kPairStages, MODE>;
    constexpr int smem = PairSmem<kPairStages>::DYN_BYTES;
    if ((st = ensure_smem_attr(info, kernel, smem)) != NVFP4LORA_OK) return st;

    static std::atomic<int> regs_ok{0};            // one per instantiation
    if ((st = check_split_regs(kernel, kPairRegsLaunch, regs_ok, "pair GEMM")) != NVFP4LORA_OK) return st;

    CUtensorMap tm_a, tm_b, tm_d, tm_lb, tm_out;
    std::memset(&tm_d, 0, sizeof(tm_d));
    std::memset(&tm_lb, 0, sizeof(tm_lb));
    std::memset(&tm_out, 0, sizeof(tm_out));
    if ((st = encode_2d(&tm_a, a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K / 2, M, 128, 128)) != NVFP4LORA_OK) return st;
    if ((st = encode_2d(&tm_b, b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K / 2, N, 128, 128)) != NVFP4LORA_OK) return st;
    if (MODE != Mode::Off) {
        if ((st = encode_2d(&tm_d, d, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, r, M, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B, kLoraPromotion)) != NVFP4LORA_OK) return st;
        // raw: per N-half, 64 of each CTA's 128 lora_b rows; prepared: all 128
        const int lb_rows = (MODE == Mode::Raw) ? 64 : 128;
        if ((st = encode_2d(&tm_lb, lb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, r, N, 64, lb_rows, CU_TENSOR_MAP_SWIZZLE_128B, kLoraPromotion)) != NVFP4LORA_OK) return st;
    }
    const bool vec_out = (N % 8 == 0 && (bias == nullptr || aligned(bias, 16)));
    if (vec_out &&
        (st = encode_2d(&tm_out, out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, N, M, kOutBoxCols, kOutBoxRows,
                        CU_TENSOR_MAP_SWIZZLE_NONE)) != NVFP4LORA_OK)
        return st;

    PairArgs args;
    args.alpha = alpha;
    args.scale = scale;
    args.a_sf = a_sf;
    args.b_sf = b_sf;
    args.bias = bias;
    args.out = out;
    args.M = (int)M;
    args.N = (int)N;
    args.K = (int)K;
    args.r = (int)r;
    args.m_pairs = (int)((M + kPairTileM - 1) / kPairTileM);
    args.n_tiles = (int)((N + kTileN - 1) / kTileN);
    const int64_t tiles = (int64_t)args.m_pairs * args.n_tiles;
    if (tiles > INT32_MAX) return fail(NVFP4LORA_ERR_INVALID_ARG, "too many output tiles (M x N too large)");
    args.num_tiles = (int)tiles;
    args.k_stages = (int)(K / 256);
    args.sf_atoms_k = (int)(K / 64);
    args.sf_row_blocks_a = (int)((M + 127) / 128);
    args.sf_row_blocks_b = (int)((N + 127) / 128);
    args.vec_out = vec_out ? 1 : 0;

    const int pairs = (int)std::min<int64_t>(tiles, info->sms / 2);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tm_a, tm_b, tm_d, tm_lb, tm_out, args);
    if (e != cudaSuccess) return cuda_fail(e, "pair GEMM launch");
    return NVFP4LORA_OK;
}

// The SM-pair kernel measured faster than the single-SM one on every shape with M >= 128 where both
// run the same number of waves (2-6 % at M = 128..384, N = 14336; 20-30 % at M >= 2048 since it
// stages scales with register stores and halves each SM's B traffic), and slower where its 256-row
// tiles add a wave (4736 x 1024 x 8192: 31.8 against 20.9 us).  It is used from M = 128 on when its
// wave count over the SM pairs is no larger than the single-SM kernel's over the SMs.
//
// One exception, measured on the raw path with a rank below 32 that is not a multiple of 16 (the
// narrow-row LoRA loads above) at M <= 256: 256 x 14336 x 4096, r = 8 ran 15.5 us on the single-SM
// kernel against 16.9 on the pair kernel (128 rows: 15.2 against 16.1), so those calls stay on the
// single-SM kernel.
bool use_pair_kernel(int64_t M, int64_t N, bool raw, int64_t r) {
    if (M < 128) return false;
    if (raw && r % 16 != 0 && r < 32 && M <= 256) return false;
    int dev = 0;
    DeviceInfo* info = nullptr;
    if (device_info(&dev, &info) != NVFP4LORA_OK) return false;
    const int64_t n_tiles = (N + kTileN - 1) / kTileN;
    const int64_t t1 = (M + kTileM - 1) / kTileM * n_tiles, t2 = (M + kPairTileM - 1) / kPairTileM * n_tiles;
    const int64_t sms = info->sms, pairs = info->sms / 2;
    return (t2 + pairs - 1) / pairs <= (t1 + sms - 1) / sms;
}

// Chooses the decode kernel for M <= 32, the SM-pair kernel where use_pair_kernel says so, and the
// single-SM tiled kernel otherwise.
template <Mode MODE>
nvfp4lora_status launch(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, const uint8_t* b_sf,
                        const float* alpha, const float* scale, const uint16_t* d, const uint16_t* lb, int64_t r,
                        const uint16_t* bias, uint16_t* out, int64_t M, int64_t N, int64_t K, cudaStream_t stream) {
    if (M <= kDecodeMaxM)
        return launch_decode<MODE>(a, b, a_sf, b_sf, alpha, scale, d, lb, r, bias, out, M, N, K, stream);
    if (use_pair_kernel(M, N, MODE == Mode::Raw, r))
        return launch_gemm_pair<MODE>(a, b, a_sf, b_sf, alpha, scale, d, lb, r, bias, out, M, N, K, stream);
    return launch_gemm<MODE>(a, b, a_sf, b_sf, alpha, scale, d, lb, r, bias, out, M, N, K, stream);
}

// ---------------------------------------------------------------------------------------
// fold launch
// ---------------------------------------------------------------------------------------

nvfp4lora_status launch_fold(const uint16_t* lora_b, const float* lora_scale, const float* alpha,
                             uint16_t* b_folded, float* ratio, int64_t N, int64_t r, cudaStream_t stream) {
    int dev = 0;
    DeviceInfo* info = nullptr;
    nvfp4lora_status st = device_info(&dev, &info);
    if (st != NVFP4LORA_OK) return st;
    const int64_t groups = N * r / 8;
    const int64_t want = (groups + kFoldThreads - 1) / kFoldThreads;
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(want, (int64_t)info->sms * 8));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kFoldThreads);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, fold_kernel, lora_b, lora_scale, alpha, b_folded, ratio, groups);
    if (e != cudaSuccess) return cuda_fail(e, "fold launch");
    return NVFP4LORA_OK;
}

nvfp4lora_status check_fold_args(const uint16_t* lora_b, const float* lora_scale, const float* alpha,
                                  int64_t N, int64_t r, const uint16_t* b_folded, const float* ratio) {
    if (N < 1) return fail(NVFP4LORA_ERR_INVALID_ARG, "N = %lld: N >= 1 is required", (long long)N);
    if (N > kMaxDim) return fail(NVFP4LORA_ERR_INVALID_ARG, "N <= 2^30 is required");
    nvfp4lora_status st = check_rank(r);
    if (st != NVFP4LORA_OK) return st;
    if (!lora_b || !lora_scale || !alpha || !b_folded || !ratio)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "lora_b, lora_scale, alpha, b_folded and ratio must be non-null");
    if (!aligned(lora_b, 16) || !aligned(b_folded, 16))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "lora_b and b_folded must be 16-byte aligned");
    if (!aligned(lora_scale, 4) || !aligned(alpha, 4) || !aligned(ratio, 4))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "lora_scale, alpha and ratio must be 4-byte aligned");
    if (ratio == lora_scale || ratio == alpha)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "ratio must not alias lora_scale or alpha");
    return NVFP4LORA_OK;
}

// ---------------------------------------------------------------------------------------
// routed tokens, 8-bit quantizers and the 8-bit product: shared launch helpers
// ---------------------------------------------------------------------------------------

// A launch with the programmatic serialization attribute: every kernel launched through it waits
// (griddepcontrol.wait) before it touches memory that an earlier kernel may write.
template <typename Kernel, typename... Args>
nvfp4lora_status launch_dependent(const char* what, Kernel kernel, int64_t grid, int block, cudaStream_t stream,
                                  const Args&... kargs) {
    if (grid > INT32_MAX) return fail(NVFP4LORA_ERR_INVALID_ARG, "%s: too large (more than 2^31 blocks)", what);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, kargs...);
    if (e != cudaSuccess) return cuda_fail(e, what);
    return NVFP4LORA_OK;
}

// Slots up to which every CTA of the permute kernel counts all of them itself (one launch).
constexpr int64_t kMoeSelfCountSlots = 4096;

nvfp4lora_status check_routing(int64_t T, int64_t top_k, int64_t rows) {
    if (T < 0 || T > kMaxDim) return fail(NVFP4LORA_ERR_INVALID_ARG, "num_tokens = %lld out of range", (long long)T);
    if (top_k < 1 || top_k > kMoeMaxTopK)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "top_k = %lld: 1 <= top_k <= %d is required", (long long)top_k, kMoeMaxTopK);
    if (T * top_k > kMaxDim) return fail(NVFP4LORA_ERR_INVALID_ARG, "num_tokens * top_k too large");
    if (rows < 0 || rows > kMaxDim) return fail(NVFP4LORA_ERR_INVALID_ARG, "padded_rows = %lld out of range", (long long)rows);
    return NVFP4LORA_OK;
}

// Two buffers share bytes (an empty or a null one shares none).
bool overlap(const void* p, int64_t np, const void* q, int64_t nq) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a && b && np > 0 && nq > 0 && a < b + (uintptr_t)nq && b < a + (uintptr_t)np;
}

// A buffer and the fp32 elements (i, j) at `base` + i * si + j * sj, i < ni, j < nj, share bytes.  Exact where one
// stride steps over all elements of the other (a matrix, its transpose, their slices), so that what lies in the gaps
// between rows is told apart; elements that interleave in another way count as all bytes from the first to the last.
bool overlap_elements(const void* p, int64_t np, const float* base, int64_t ni, int64_t si, int64_t nj, int64_t sj) {
    using Wide = __int128;                       // strides are the caller's: no product of them overflows
    if (!p || !base || np <= 0 || ni <= 0 || nj <= 0) return false;
    if (ni == 1) si = 0;
    if (nj == 1) sj = 0;
    if (si < sj) { std::swap(si, sj); std::swap(ni, nj); }           // i: the outer dimension
    Wide lo = (Wide)reinterpret_cast<uintptr_t>(p) - (Wide)reinterpret_cast<uintptr_t>(base), hi = lo + np;
    // the first and the last of n pieces of `size` bytes, `step` apart, that [lo, hi) may share bytes with
    auto pieces = [&](Wide n, Wide step, Wide size, Wide& first, Wide& last) {
        auto floor_div = [](Wide a, Wide b) { return a >= 0 ? a / b : -((-a + b - 1) / b); };
        first = step == 0 ? 0 : std::max<Wide>(0, floor_div(lo - size, step) + 1);
        last = step == 0 ? 0 : std::min<Wide>(n - 1, floor_div(hi - 1, step));
        return first <= last && lo < last * step + size && hi > first * step;
    };
    const Wide inner = 4 * ((Wide)(nj - 1) * sj + 1);
    Wide first = 0, last = 0;
    if (lo >= inner + 4 * (Wide)(ni - 1) * si || hi <= 0) return false;
    if (ni > 1 && 4 * (Wide)si < inner) return true;
    if (!pieces(ni, 4 * (Wide)si, inner, first, last)) return false;
    if (first < last) return true;               // two rows' bytes: the second's first element lies between
    lo -= first * 4 * si;
    hi -= first * 4 * si;
    return pieces(nj, 4 * (Wide)sj, 4, first, last);
}

// A contiguous buffer of a call, and fp32 scales of any strides.
struct Span {
    const char* name;
    const void* p;
    int64_t bytes;
};
struct Scales {
    const char* name;
    const float* p;
    int64_t rows, stride_row, cols, stride_col;
};

// Blocks write their results while others still read: nothing that a call writes may share a byte with what it
// reads, nor two of its results with each other.
nvfp4lora_status check_apart(std::initializer_list<Span> written, std::initializer_list<Span> read) {
    for (const Span* w = written.begin(); w != written.end(); ++w) {
        for (const Span& r : read)
            if (overlap(w->p, w->bytes, r.p, r.bytes))
                return fail(NVFP4LORA_ERR_INVALID_ARG, "%s must not overlap %s", w->name, r.name);
        for (const Span* v = w + 1; v != written.end(); ++v)
            if (overlap(w->p, w->bytes, v->p, v->bytes))
                return fail(NVFP4LORA_ERR_INVALID_ARG, "%s must not overlap %s", w->name, v->name);
    }
    return NVFP4LORA_OK;
}

nvfp4lora_status check_apart(const Scales& s, std::initializer_list<Span> others) {
    for (const Span& o : others)
        if (overlap_elements(o.p, o.bytes, s.p, s.rows, s.stride_row, s.cols, s.stride_col))
            return fail(NVFP4LORA_ERR_INVALID_ARG, "%s must not overlap %s", s.name, o.name);
    return NVFP4LORA_OK;
}

bool valid_type(int32_t t) {
    return t == NVFP4LORA_DTYPE_BF16 || t == NVFP4LORA_DTYPE_FP16 || t == NVFP4LORA_DTYPE_FP32;
}

int type_bytes(int32_t t) { return t == NVFP4LORA_DTYPE_FP32 ? 4 : 2; }

// The element type of a row operator as a template argument.
template <typename F>
nvfp4lora_status by_type(int32_t t, F f) {
    if (t == NVFP4LORA_DTYPE_BF16) return f(std::integral_constant<MoeType, MoeType::BF16>{});
    if (t == NVFP4LORA_DTYPE_FP16) return f(std::integral_constant<MoeType, MoeType::FP16>{});
    return f(std::integral_constant<MoeType, MoeType::FP32>{});
}

bool rows_aligned16(int64_t row_bytes, std::initializer_list<const void*> ptrs) {
    if (row_bytes % 16 != 0) return false;
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return false;
    return true;
}

nvfp4lora_status check_scale_strides(int64_t rows, int64_t groups, int64_t sr, int64_t sg) {
    // an output: no two elements may share an address
    const bool row_major = sg >= 1 && (rows <= 1 || sr >= (groups - 1) * sg + 1);
    const bool col_major = sr >= 1 && (groups <= 1 || sg >= (rows - 1) * sr + 1);
    if (!(row_major || col_major) || sr < 0 || sg < 0)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "scales strides (%lld, %lld): row-major or column-major elements that do "
                    "not overlap are required", (long long)sr, (long long)sg);
    return NVFP4LORA_OK;
}

nvfp4lora_status check_fp8_rows(const void* x, const uint8_t* q, const float* scales, int64_t rows, int64_t H,
                                int32_t dtype) {
    if (rows < 1 || H < 1) return fail(NVFP4LORA_ERR_INVALID_ARG, "rows >= 1 and H >= 1 are required (rows=%lld H=%lld)",
                                       (long long)rows, (long long)H);
    if (rows > kMaxDim || H > kMaxK) return fail(NVFP4LORA_ERR_INVALID_ARG, "rows <= 2^30 and H <= 2^20 are required");
    if (!valid_type(dtype)) return fail(NVFP4LORA_ERR_INVALID_ARG, "dtype must be NVFP4LORA_DTYPE_BF16, _FP16 or _FP32");
    if (!x || !q || !scales) return fail(NVFP4LORA_ERR_INVALID_ARG, "x, q and scales must be non-null");
    if (!aligned(x, type_bytes(dtype)) || !aligned(scales, 4))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "x must be aligned to its elements and scales 4-byte aligned");
    return NVFP4LORA_OK;
}

// ---- the 8-bit product ----

template <OutType OT, int TN>
nvfp4lora_status launch_fp8_pair(DeviceInfo* info, const uint8_t* a, const uint8_t* b, Fp8GemmArgs args, int64_t K,
                                 cudaStream_t stream) {
    nvfp4lora_status st;
    auto kernel = fp8_gemm_pair_kernel<OT, TN>;
    constexpr int smem = Fp8Smem<TN>::DYN_BYTES;
    if ((st = ensure_smem_attr(info, kernel, smem)) != NVFP4LORA_OK) return st;
    if constexpr (TN == 256) {
        static std::atomic<int> regs_ok{0};        // one per instantiation
        if ((st = check_split_regs(kernel, kFp8RegsLaunch, regs_ok, "8-bit product")) != NVFP4LORA_OK) return st;
    }
    CUtensorMap tm_a, tm_b, tm_out;
    std::memset(&tm_out, 0, sizeof(tm_out));
    if ((st = encode_2d(&tm_a, a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K, args.M, 128, 128)) != NVFP4LORA_OK) return st;
    if ((st = encode_2d(&tm_b, b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K, args.N, 128, TN / 2)) != NVFP4LORA_OK) return st;
    constexpr int esize = OT == OutType::FP32 ? 4 : 2;
    args.out_bytes = 16;
    while (((int64_t)args.N * esize) % args.out_bytes != 0 || !aligned(args.out, args.out_bytes)) args.out_bytes /= 2;
    if (args.out_bytes == 16 &&
        (st = encode_2d(&tm_out, args.out,
                        OT == OutType::FP32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                            : OT == OutType::FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                        esize, args.N, args.M, 64 / esize, kFp8BoxRows, CU_TENSOR_MAP_SWIZZLE_64B)) != NVFP4LORA_OK)
        return st;
    args.m_tiles = (args.M + kFp8TileM - 1) / kFp8TileM;
    args.n_tiles = (args.N + TN - 1) / TN;
    const int64_t tiles = (int64_t)args.m_tiles * args.n_tiles;
    if (tiles > INT32_MAX - info->sms)       // a tile index one wave past the last stays in int32
        return fail(NVFP4LORA_ERR_INVALID_ARG, "too many output tiles (M x N too large)");
    args.num_tiles = (int)tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)std::min<int64_t>(tiles, info->sms / 2));
    cfg.blockDim = dim3(kFp8Threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tm_a, tm_b, tm_out, args);
    if (e != cudaSuccess) return cuda_fail(e, "8-bit product launch");
    return NVFP4LORA_OK;
}

template <int MT, OutType OT>
nvfp4lora_status launch_fp8_splitk(DeviceInfo* info, const uint8_t* a, const uint8_t* b, const Fp8SplitArgs& args,
                                   int64_t K, cudaStream_t stream) {
    nvfp4lora_status st;
    auto kernel = fp8_splitk_kernel<MT, OT>;
    constexpr int smem = Fp8SplitPlan<MT>::DYN_BYTES;
    if ((st = ensure_smem_attr(info, kernel, smem)) != NVFP4LORA_OK) return st;
    CUtensorMap tm_a, tm_b;
    if ((st = encode_2d(&tm_a, a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K, args.M, 128, MT)) != NVFP4LORA_OK) return st;
    if ((st = encode_2d(&tm_b, b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K, args.N, 128, 128)) != NVFP4LORA_OK) return st;
    const int64_t m_tiles = (args.M + MT - 1) / MT;
    if (m_tiles > 65535) return fail(NVFP4LORA_ERR_INVALID_ARG, "too many output tiles (M too large)");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((args.N + 127) / 128), (unsigned)args.splits, (unsigned)m_tiles);
    cfg.blockDim = dim3(Fp8SplitPlan<MT>::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (args.splits > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 1;
        attr[1].val.clusterDim.y = args.splits;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tm_a, tm_b, args);
    if (e != cudaSuccess) return cuda_fail(e, "8-bit product launch (split K)");
    return NVFP4LORA_OK;
}

struct Fp8Plan {
    bool pair;               // the SM-pair kernel
    int mt, splits;          // the split-K kernel's token tile and cluster size
    int tn;                  // the SM-pair kernel's tile columns
};

// The kernel of a shape.  Split-K kernel: the token tile is the smallest that holds M (128 from 65 rows on);
// K is split over clusters of a power of two of CTAs (3, 5, 6 and 7 measured slower than the power below:
// clusters of those sizes fill the GPU's processor clusters badly) while all CTAs are resident at once (a
// second wave always lost: 64 x 8192 x 4096 12.2 us with 4-way clusters, 19.4 with 5) and either SMs are free or
// a CTA still has 16 blocks to stream (16 x 4096 x 4096: 7.0 us 4-way, 7.4 8-way; 16 x 4096 x 14336: 14.3 and 13.2).
// With 128-token tiles the SM-pair kernel takes what cannot be split (300 x 4096 x 4096: 13.7 us against 19.6 unsplit;
// N x 8192 with N = 10240: 65 rows 32.2 against 33.7, 128 32.9 and 35.3, 256 33.4 and 69; N = 28672: 60.9 and 70, 63
// and 74, 67 and 150), and what can be split only 2-way over fewer than 48 blocks: its time per block of K is the lower,
// 2-way splits halve the blocks.  Pair against 2-way over 16, 32, 48, 64 and 112 blocks: 128 x 5120 9.0 and 11.2, 13.9
// and 15.2, 18.8 and 18.9, 23.7 and 22.6, 38.2 and 34.3 us; 128 x 9472 9.8 and 12.0, 14.7 and 15.9, 19.6 and 19.7, 24.9
// and 24.0, 40.9 and 37.9; 256 x 4096 8.7 and 11.4, 13.4 and 15.1, 18.0 and 18.7, 22.6 and 22.4, 36.5 and 33.6.  (128 x
// 4096 x 4096, 4-way: 13.9 on the pair against 11.7.)  Its tiles are 128 columns wide while they fit the GPU in one wave (512 x 4096 x 4096: 14.8 us
// against 19.6 with 256; 1536 x 2048 x 4096, 96 tiles of 128: 25.7 against 21.0).
Fp8Plan plan_fp8(int64_t M, int64_t N, int64_t kblocks, int sms) {
    Fp8Plan p{false, M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128, 1, 256};
    const int64_t tiles = (N + 127) / 128 * ((M + p.mt - 1) / p.mt);
    const int64_t slots = p.mt <= 64 ? 2 * (int64_t)sms : sms;
    while (2 * p.splits <= kSplitMaxS && 2 * p.splits <= kblocks && 2 * p.splits * tiles <= slots &&
           (2 * p.splits * tiles <= sms || kblocks / p.splits >= 16))
        p.splits *= 2;
    p.pair = p.mt == 128 && (p.splits == 1 || (p.splits == 2 && kblocks < 48));
    if ((M + kFp8TileM - 1) / kFp8TileM * ((N + 127) / 128) <= sms / 2) p.tn = 128;
    return p;
}

template <OutType OT>
nvfp4lora_status launch_fp8(DeviceInfo* info, const uint8_t* a, const uint8_t* b, const Fp8GemmArgs& g, int64_t K,
                            cudaStream_t stream) {
    const Fp8Plan plan = plan_fp8(g.M, g.N, g.kblocks, info->sms);
    if (plan.pair) return plan.tn == 128 ? launch_fp8_pair<OT, 128>(info, a, b, g, K, stream)
                                         : launch_fp8_pair<OT, 256>(info, a, b, g, K, stream);
    Fp8SplitArgs s;
    s.a_scale = g.a_scale;
    s.b_scale = g.b_scale;
    s.bias = g.bias;
    s.out = g.out;
    s.stride_am = g.stride_am;
    s.stride_ak = g.stride_ak;
    s.M = g.M;
    s.N = g.N;
    s.kblocks = g.kblocks;
    s.splits = plan.splits;
    constexpr int esize = OT == OutType::FP32 ? 4 : 2;
    s.vec_out = g.N % 4 == 0 && aligned(g.out, 4 * esize);
    switch (plan.mt) {
        case 16: return launch_fp8_splitk<16, OT>(info, a, b, s, K, stream);
        case 32: return launch_fp8_splitk<32, OT>(info, a, b, s, K, stream);
        case 64: return launch_fp8_splitk<64, OT>(info, a, b, s, K, stream);
        default: return launch_fp8_splitk<128, OT>(info, a, b, s, K, stream);
    }
}

}  // namespace
}  // namespace nvfp4lora

using namespace nvfp4lora;

extern "C" {

nvfp4lora_status nvfp4lora_mm(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, int64_t a_sf_bytes,
                              const uint8_t* b_sf, int64_t b_sf_bytes, const float* alpha,
                              const uint16_t* d, const uint16_t* lora_b, const float* lora_scale, int64_t r,
                              const uint16_t* bias, uint16_t* out, int64_t M, int64_t N, int64_t K,
                              nvfp4lora_stream stream) {
    t_last_error.clear();
    nvfp4lora_status st = check_base(a, b, a_sf, a_sf_bytes, b_sf, b_sf_bytes, alpha, bias, out, M, N, K);
    if (st != NVFP4LORA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (lora_scale == nullptr)
        return launch<Mode::Off>(a, b, a_sf, b_sf, alpha, nullptr, nullptr, nullptr, 0, bias, out, M, N, K, s);
    if ((st = check_rank(r)) != NVFP4LORA_OK) return st;
    if (!d || !lora_b) return fail(NVFP4LORA_ERR_INVALID_ARG, "lora_scale given: d and lora_b must be non-null");
    if (!aligned(d, 16) || !aligned(lora_b, 16))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "d and lora_b must be 16-byte aligned");
    if (!aligned(lora_scale, 4)) return fail(NVFP4LORA_ERR_INVALID_ARG, "lora_scale must be 4-byte aligned");
    return launch<Mode::Raw>(a, b, a_sf, b_sf, alpha, lora_scale, d, lora_b, r, bias, out, M, N, K, s);
}

nvfp4lora_status nvfp4lora_prepare(const uint16_t* lora_b, const float* lora_scale, const float* alpha,
                                   int64_t N, int64_t r, uint16_t* b_folded, float* ratio,
                                   uint64_t src_version, nvfp4lora_adapter* adapter_out,
                                   nvfp4lora_stream stream) {
    t_last_error.clear();
    if (!adapter_out) return fail(NVFP4LORA_ERR_INVALID_ARG, "adapter_out must be non-null");
    nvfp4lora_status st = check_fold_args(lora_b, lora_scale, alpha, N, r, b_folded, ratio);
    if (st != NVFP4LORA_OK) return st;
    int dev = 0;
    DeviceInfo* info = nullptr;
    if ((st = device_info(&dev, &info)) != NVFP4LORA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // The single host read of the adapter switch: (lora_scale, alpha).
    float host[2] = {0.0f, 0.0f};
    cudaError_t e = cudaMemcpyAsync(&host[0], lora_scale, sizeof(float), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaMemcpyAsync(&host[1], alpha, sizeof(float), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "reading lora_scale and alpha");
    if (host[1] == 0.0f)
        return fail(NVFP4LORA_ERR_ALPHA_ZERO, "alpha == 0: lora_scale / alpha is undefined "
                                              "(the alpha == 0 LoRA-only call is the raw path)");
    volatile float q = host[0] / host[1];
    if (!std::isfinite((float)q))
        return fail(NVFP4LORA_ERR_ALPHA_ZERO, "lora_scale / alpha = %g is not finite", (double)q);
    if ((st = launch_fold(lora_b, lora_scale, alpha, b_folded, ratio, N, r, s)) != NVFP4LORA_OK) return st;
    adapter_out->b_folded = b_folded;
    adapter_out->ratio = ratio;
    adapter_out->alpha = alpha;
    adapter_out->lora_b = lora_b;
    adapter_out->lora_scale = lora_scale;
    adapter_out->N = N;
    adapter_out->r = r;
    adapter_out->src_version = src_version;
    adapter_out->device = dev;
    adapter_out->reserved = 0;
    return NVFP4LORA_OK;
}

nvfp4lora_status nvfp4lora_refold(nvfp4lora_adapter* adapter, const uint16_t* lora_b, const float* lora_scale,
                                  const float* alpha, int64_t N, int64_t r, uint64_t src_version,
                                  nvfp4lora_stream stream) {
    t_last_error.clear();
    if (!adapter) return fail(NVFP4LORA_ERR_INVALID_ARG, "adapter must be non-null");
    nvfp4lora_status st = check_fold_args(lora_b, lora_scale, alpha, N, r, adapter->b_folded, adapter->ratio);
    if (st != NVFP4LORA_OK) return st;
    if (alpha != adapter->alpha)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "alpha must be the adapter's own alpha tensor");
    if (N != adapter->N || r != adapter->r)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "lora_b must keep the adapter's [N, r] = [%lld, %lld]",
                    (long long)adapter->N, (long long)adapter->r);
    int dev = 0;
    DeviceInfo* info = nullptr;
    if ((st = device_info(&dev, &info)) != NVFP4LORA_OK) return st;
    if (dev != adapter->device)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "lora_b must stay on the adapter's device %d", adapter->device);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if ((st = launch_fold(lora_b, lora_scale, alpha, adapter->b_folded, adapter->ratio, N, r, s)) != NVFP4LORA_OK)
        return st;
    adapter->lora_b = lora_b;
    adapter->lora_scale = lora_scale;
    adapter->src_version = src_version;
    return NVFP4LORA_OK;
}

nvfp4lora_status nvfp4lora_mm_prepared(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, int64_t a_sf_bytes,
                                       const uint8_t* b_sf, int64_t b_sf_bytes, const float* alpha,
                                       const uint16_t* d, const nvfp4lora_adapter* adapter,
                                       const uint16_t* cur_lora_b, const float* cur_lora_scale,
                                       uint64_t cur_src_version, const uint16_t* bias, uint16_t* out,
                                       int64_t M, int64_t N, int64_t K, nvfp4lora_stream stream) {
    t_last_error.clear();
    nvfp4lora_status st = check_base(a, b, a_sf, a_sf_bytes, b_sf, b_sf_bytes, alpha, bias, out, M, N, K);
    if (st != NVFP4LORA_OK) return st;
    if (!adapter) return fail(NVFP4LORA_ERR_INVALID_ARG, "adapter must be non-null");
    if (!adapter->b_folded || !adapter->ratio)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "adapter has no b_folded / ratio buffers");
    if (adapter->N != N)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "adapter has N = %lld, the call N = %lld",
                    (long long)adapter->N, (long long)N);
    if ((st = check_rank(adapter->r)) != NVFP4LORA_OK) return st;
    if (!d) return fail(NVFP4LORA_ERR_INVALID_ARG, "the prepared path still requires d");
    if (!aligned(d, 16) || !aligned(adapter->b_folded, 16))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "d and b_folded must be 16-byte aligned");
    if (alpha != adapter->alpha)
        return fail(NVFP4LORA_ERR_STALE_ADAPTER,
                    "the adapter was prepared for another alpha tensor; re-prepare when alpha changes");
    if (cur_lora_b != adapter->lora_b || cur_lora_scale != adapter->lora_scale)
        return fail(NVFP4LORA_ERR_STALE_ADAPTER, "the adapter's lora_b / lora_scale moved since the prepare");
    if (cur_src_version != adapter->src_version)
        return fail(NVFP4LORA_ERR_STALE_ADAPTER, "the adapter's lora_b / lora_scale were written since the prepare");
    int dev = 0;
    DeviceInfo* info = nullptr;
    if ((st = device_info(&dev, &info)) != NVFP4LORA_OK) return st;
    if (dev != adapter->device)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "the adapter lives on device %d, the call runs on %d",
                    adapter->device, dev);
    return launch<Mode::Prepared>(a, b, a_sf, b_sf, alpha, adapter->ratio, d, adapter->b_folded,
                                       adapter->r, bias, out, M, N, K, reinterpret_cast<cudaStream_t>(stream));
}

nvfp4lora_status nvfp4lora_grouped_mm(const uint8_t* a, const uint8_t* b, const uint8_t* a_sf, int64_t a_sf_bytes,
                                      const uint8_t* b_sf, int64_t b_sf_bytes, const int32_t* m_indptr,
                                      int64_t num_experts, const float* alpha, const uint16_t* d,
                                      const uint16_t* lora_b, const float* lora_scale, int64_t r,
                                      const uint16_t* bias, uint16_t* out, int64_t rows, int64_t N, int64_t K,
                                      nvfp4lora_stream stream) {
    t_last_error.clear();
    if (num_experts < 1 || num_experts > kMaxExperts)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "num_experts = %lld: 1 <= num_experts <= %d is required",
                    (long long)num_experts, kMaxExperts);
    if (rows > kMaxDim || (int64_t)num_experts * N > kMaxDim)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "rows and num_experts x N must be at most 2^30");
    // the per-expert scale buffers of b are consecutive, ceil(N/128)*128*K/16 bytes each
    const int64_t per_expert_sf = (N + 127) / 128 * 128 * (K / 16);
    nvfp4lora_status st = check_base(a, b, a_sf, a_sf_bytes, b_sf, per_expert_sf, alpha, bias, out, rows, N, K);
    if (st != NVFP4LORA_OK) return st;
    if (b_sf_bytes < num_experts * per_expert_sf)
        return fail(NVFP4LORA_ERR_INVALID_ARG,
                    "b_sf has %lld bytes; num_experts consecutive 128x4 buffers of N rows need %lld",
                    (long long)b_sf_bytes, (long long)(num_experts * per_expert_sf));
    if (!m_indptr || !aligned(m_indptr, 4))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "m_indptr must be a non-null, 4-byte aligned int32 array");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (lora_scale == nullptr)
        return launch_gemm_grouped<Mode::Off>(a, b, a_sf, b_sf, m_indptr, num_experts, alpha, nullptr, nullptr,
                                              nullptr, 0, bias, out, rows, N, K, s);
    if ((st = check_rank(r)) != NVFP4LORA_OK) return st;
    if (!d || !lora_b) return fail(NVFP4LORA_ERR_INVALID_ARG, "lora_scale given: d and lora_b must be non-null");
    if (!aligned(d, 16) || !aligned(lora_b, 16))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "d and lora_b must be 16-byte aligned");
    if (!aligned(lora_scale, 4)) return fail(NVFP4LORA_ERR_INVALID_ARG, "lora_scale must be 4-byte aligned");
    return launch_gemm_grouped<Mode::Raw>(a, b, a_sf, b_sf, m_indptr, num_experts, alpha, lora_scale, d, lora_b, r,
                                          bias, out, rows, N, K, s);
}

nvfp4lora_status nvfp4lora_device_status(nvfp4lora_stream stream) {
    t_last_error.clear();
    cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
    int word = 0;
    e = cudaMemcpyFromSymbol(&word, g_device_error, sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e, "reading the device error word");
    if (word != 0) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int));
        if (e != cudaSuccess) return cuda_fail(e, "clearing the device error word");
        if (word == kErrBadIndptr)
            return fail(NVFP4LORA_ERR_INVALID_ARG,
                        "grouped call: m_indptr must start at 0, be non-decreasing, hold multiples of 128 and "
                        "end at most at the row count (no tile was computed)");
        if (word == kErrBadRoute)
            return fail(NVFP4LORA_ERR_INVALID_ARG,
                        "LoRA delta: a routing entry was out of range (expert id outside [0, num_experts), "
                        "permuted index past the activation rows, or a null or misaligned bank address); "
                        "that slot was skipped");
        if (word == kErrBadSlot)
            return fail(NVFP4LORA_ERR_INVALID_ARG,
                        "routed tokens: an expert id was not below num_experts, or a permuted index not below the row "
                        "count; that slot was left out");
        return fail(NVFP4LORA_ERR_DEVICE_TIMEOUT, "a kernel's bounded wait ran out (pipeline stalled)");
    }
    return NVFP4LORA_OK;
}

nvfp4lora_status nvfp4lora_selftest_wait_timeout(int64_t limit_ns, nvfp4lora_stream stream) {
    t_last_error.clear();
    if (limit_ns <= 0 || limit_ns > 1000000000)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "limit_ns = %lld: 0 < limit_ns <= 1e9 is required", (long long)limit_ns);
    int dev = 0;
    DeviceInfo* info = nullptr;
    nvfp4lora_status st = device_info(&dev, &info);
    if (st != NVFP4LORA_OK) return st;
    wait_timeout_selftest_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        (unsigned long long)limit_ns);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "self-test launch");
    return NVFP4LORA_OK;
}

nvfp4lora_status nvfp4lora_quantize(const uint16_t* x, int64_t rows, int64_t K, const float* global_scale,
                                    uint8_t* codes, uint8_t* scales, int64_t scales_bytes, nvfp4lora_stream stream) {
    t_last_error.clear();
    if (!x || !global_scale || !codes || !scales)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "x, global_scale, codes and scales must be non-null");
    if (rows < 1 || K < 64 || K % 64 != 0)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "rows >= 1 and K >= 64 with K %% 64 == 0 are required (rows=%lld K=%lld)",
                    (long long)rows, (long long)K);
    if (rows > (int64_t)1 << 40 || K > (int64_t)1 << 30)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "rows x K too large");
    const int64_t need = (rows + 127) / 128 * 128 * (K / 16);
    if (scales_bytes < need)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "scales needs %lld bytes (rows padded to 128 x K/16), got %lld",
                    (long long)need, (long long)scales_bytes);
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "x, codes and scales must be 16-byte aligned");
    if (!aligned(global_scale, 4)) return fail(NVFP4LORA_ERR_INVALID_ARG, "global_scale must be 4-byte aligned");
    int dev = 0;
    DeviceInfo* info = nullptr;
    nvfp4lora_status st = device_info(&dev, &info);
    if (st != NVFP4LORA_OK) return st;
    const int64_t total = (rows + 127) / 128 * 128 * (K / 16);             // one thread per block per step
    const int64_t want = (total + kQuantThreads - 1) / kQuantThreads;
    // a grid-stride loop over one wave: the launch bounds keep 8 CTAs resident per SM
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(want, (int64_t)info->sms * 8));
    quantize_kernel<<<grid, kQuantThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(x, rows, K, global_scale,
                                                                                          codes, scales);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "quantize launch");
    return NVFP4LORA_OK;
}

nvfp4lora_status nvfp4lora_bgmv_moe_gemm2_lora_delta(
    const void* act, int64_t padded_rows, int64_t I, const int32_t* perm, const int64_t* w_ptr_a,
    int64_t lora_stride_a, const int64_t* w_ptr_b, int64_t lora_stride_b, const int32_t* topk_ids,
    const float* topk_weights, const int32_t* lora_ids, int64_t num_tokens, int64_t top_k, int64_t num_experts,
    int64_t rank, int64_t hidden_size, int32_t lora_dtype, float scale, int32_t out_dtype, void* out,
    nvfp4lora_stream stream) {
    t_last_error.clear();
    const int64_t kMaxDim = (int64_t)1 << 30;
    if (num_tokens < 0 || num_tokens > kMaxDim)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "num_tokens = %lld out of range", (long long)num_tokens);
    if (top_k < 1 || top_k > kBgmvMaxTopK)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "top_k = %lld: 1 <= top_k <= %d is required", (long long)top_k,
                    kBgmvMaxTopK);
    if (rank < 8 || rank > kBgmvMaxRank || rank % 8 != 0)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "rank = %lld: 8 <= rank <= %d with rank %% 8 == 0 is required",
                    (long long)rank, kBgmvMaxRank);
    if (I < 8 || I % 8 != 0 || I > kMaxDim)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "I = %lld: I >= 8 with I %% 8 == 0 is required", (long long)I);
    if (hidden_size < 1 || hidden_size > kMaxDim)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "hidden_size = %lld out of range", (long long)hidden_size);
    if (num_experts < 1 || num_experts > kMaxDim)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "num_experts = %lld out of range", (long long)num_experts);
    if (padded_rows < 0 || padded_rows > kMaxDim)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "padded_rows = %lld out of range", (long long)padded_rows);
    if (num_tokens * top_k > kMaxDim)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "num_tokens * top_k too large");
    if (lora_stride_a < 0 || lora_stride_b < 0 || lora_stride_a % 8 != 0 || lora_stride_b % 8 != 0)
        return fail(NVFP4LORA_ERR_INVALID_ARG,
                    "lora_stride_a = %lld, lora_stride_b = %lld: non-negative multiples of 8 are required "
                    "(adapter blocks start on 16-byte boundaries)", (long long)lora_stride_a, (long long)lora_stride_b);
    if ((lora_dtype != NVFP4LORA_DTYPE_BF16 && lora_dtype != NVFP4LORA_DTYPE_FP16) ||
        (out_dtype != NVFP4LORA_DTYPE_BF16 && out_dtype != NVFP4LORA_DTYPE_FP16))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "lora_dtype and out_dtype must be NVFP4LORA_DTYPE_BF16 or _FP16");
    if (num_tokens == 0) return NVFP4LORA_OK;
    if (!perm || !w_ptr_a || !w_ptr_b || !topk_ids || !topk_weights || !lora_ids || !out ||
        (!act && padded_rows > 0))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "every pointer argument must be non-null");
    if (!aligned(act, 16)) return fail(NVFP4LORA_ERR_INVALID_ARG, "act must be 16-byte aligned");
    if (!aligned(w_ptr_a, 8) || !aligned(w_ptr_b, 8))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "w_ptr_a and w_ptr_b must be 8-byte aligned");
    if (!aligned(perm, 4) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4) || !aligned(lora_ids, 4) ||
        !aligned(out, 2))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "routing tables must be 4-byte aligned and out 2-byte aligned");
    int dev = 0;
    DeviceInfo* info = nullptr;
    nvfp4lora_status st = device_info(&dev, &info);
    if (st != NVFP4LORA_OK) return st;

    // A cluster of cs CTAs per token splits I (shrink) and H (expand): the smallest power of two
    // that gives about two CTAs per SM, capped by the cluster limit and by I / 8 and H; raised
    // further if one CTA's shared memory (the shrink's cells for its I slice) would not fit.
    const int64_t len = top_k * rank;
    auto fits = [&](int64_t c) { return bgmv_smem_floats(len, (I / 8 + c - 1) / c, c) * 4 <= kBgmvSmemLimit; };
    auto can_grow = [&](int64_t c) { return c < kBgmvMaxCluster && 2 * c <= I / 8 && 2 * c <= hidden_size; };
    int cs = 1;
    while (can_grow(cs) && num_tokens * cs < 2 * (int64_t)info->sms) cs *= 2;
    while (!fits(cs) && can_grow(cs)) cs *= 2;
    if (!fits(cs))
        return fail(NVFP4LORA_ERR_INVALID_ARG,
                    "top_k * rank * I too large: one CTA's share (I / %d columns, %lld rows of the adapters) needs more "
                    "than %d bytes of shared memory", cs, (long long)len, kBgmvSmemLimit);
    BgmvArgs args;
    args.act = act;
    args.perm = perm;
    args.w_ptr_a = w_ptr_a;
    args.w_ptr_b = w_ptr_b;
    args.topk_ids = topk_ids;
    args.topk_w = topk_weights;
    args.lora_ids = lora_ids;
    args.out = out;
    args.stride_a = lora_stride_a;
    args.stride_b = lora_stride_b;
    args.rows = (int)padded_rows;
    args.I = (int)I;
    args.top_k = (int)top_k;
    args.num_experts = (int)num_experts;
    args.rank = (int)rank;
    args.H = (int)hidden_size;
    args.cs = cs;
    args.scale = scale;
    const int smem = (int)(bgmv_smem_floats(len, (I / 8 + cs - 1) / cs, cs) * (int64_t)sizeof(float));

    auto pick = [&](auto kernel) -> nvfp4lora_status {
        // the delta's shared memory can exceed the 48 KB default; the L1 carve-out stays the
        // driver's choice (the activation rows are re-read through L1)
        nvfp4lora_status sa = ensure_smem_attr(info, kernel, kBgmvSmemLimit, false);
        if (sa != NVFP4LORA_OK) return sa;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(num_tokens * cs));
        cfg.blockDim = dim3(kBgmvThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = reinterpret_cast<cudaStream_t>(stream);
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cs > 1) {
            attr[1].id = cudaLaunchAttributeClusterDimension;
            attr[1].val.clusterDim.x = cs;
            attr[1].val.clusterDim.y = 1;
            attr[1].val.clusterDim.z = 1;
            cfg.numAttrs = 2;
        }
        cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args);
        if (e != cudaSuccess) return cuda_fail(e, "LoRA delta launch");
        return NVFP4LORA_OK;
    };
    const bool f16_in = lora_dtype == NVFP4LORA_DTYPE_FP16, f16_out = out_dtype == NVFP4LORA_DTYPE_FP16;
    if (f16_in)
        return f16_out ? pick(bgmv_delta_kernel<true, true>) : pick(bgmv_delta_kernel<true, false>);
    return f16_out ? pick(bgmv_delta_kernel<false, true>) : pick(bgmv_delta_kernel<false, false>);
}

nvfp4lora_status nvfp4lora_moe_permute(const void* x, int64_t num_tokens, int64_t row_bytes, const int32_t* topk_ids,
                                       int64_t top_k, int64_t num_experts, int64_t align, int32_t zero_padding,
                                       void* rows, int64_t padded_rows, int32_t* m_indptr,
                                       int32_t* expanded_idx_to_permuted_idx, int32_t* permuted_idx_to_expanded_idx,
                                       void* workspace, int64_t workspace_bytes, nvfp4lora_stream stream) {
    t_last_error.clear();
    nvfp4lora_status st = check_routing(num_tokens, top_k, padded_rows);
    if (st != NVFP4LORA_OK) return st;
    if (num_experts < 1 || num_experts > kMoeMaxExperts)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "num_experts = %lld: 1 <= num_experts <= %d is required",
                    (long long)num_experts, kMoeMaxExperts);
    if (align < 1 || align > kMoeMaxAlign)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "align = %lld: 1 <= align <= %d is required", (long long)align, kMoeMaxAlign);
    if (row_bytes < 1 || row_bytes > kMaxDim)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "row_bytes = %lld out of range", (long long)row_bytes);
    const int64_t n = num_tokens * top_k;
    const int64_t need = (n + std::min(num_experts, n) * (align - 1)) / align * align;
    if (padded_rows < need)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "padded_rows = %lld: %lld tokens, top_k = %lld, %lld experts and align = %lld "
                    "can need %lld", (long long)padded_rows, (long long)num_tokens, (long long)top_k,
                    (long long)num_experts, (long long)align, (long long)need);
    if (!m_indptr || !aligned(m_indptr, 4))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "m_indptr must be a non-null, 4-byte aligned int32 array");
    if (n > 0 && (!x || !topk_ids || !rows || !expanded_idx_to_permuted_idx))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "x, topk_ids, rows and the tables must be non-null");
    if (padded_rows > 0 && !permuted_idx_to_expanded_idx)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "permuted_idx_to_expanded_idx must be non-null");
    if (!aligned(topk_ids, 4) || !aligned(expanded_idx_to_permuted_idx, 4) || !aligned(permuted_idx_to_expanded_idx, 4))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "topk_ids and the tables must be 4-byte aligned");
    const bool counted = n > kMoeSelfCountSlots;
    const int64_t ws = counted ? (int64_t)kMoeCountChunks * num_experts * 4 : 0;
    if (counted && (!workspace || workspace_bytes < ws || !aligned(workspace, 4)))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "workspace needs %lld bytes, 4-byte aligned (got %lld)", (long long)ws,
                    (long long)workspace_bytes);
    if ((st = check_apart({{"rows", rows, padded_rows * row_bytes}, {"m_indptr", m_indptr, (num_experts + 1) * 4},
                           {"expanded_idx_to_permuted_idx", expanded_idx_to_permuted_idx, n * 4},
                           {"permuted_idx_to_expanded_idx", permuted_idx_to_expanded_idx, padded_rows * 4},
                           {"workspace", workspace, ws}},
                          {{"x", x, num_tokens * row_bytes}, {"topk_ids", topk_ids, n * 4}})) != NVFP4LORA_OK)
        return st;
    int dev = 0;
    DeviceInfo* info = nullptr;
    if ((st = device_info(&dev, &info)) != NVFP4LORA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    PermuteArgs a;
    a.x = static_cast<const uint8_t*>(x);
    a.ids = topk_ids;
    a.rows = static_cast<uint8_t*>(rows);
    a.indptr = m_indptr;
    a.idx = expanded_idx_to_permuted_idx;
    a.inv = permuted_idx_to_expanded_idx;
    a.counts = nullptr;
    a.chunk = (n + kMoeCountChunks - 1) / kMoeCountChunks;
    a.n = n;
    a.row_bytes = row_bytes;
    a.T = (int)num_tokens;
    a.top_k = (int)top_k;
    a.E = (int)num_experts;
    a.align = (int)align;
    a.capacity = (int)padded_rows;
    a.zero_padding = zero_padding != 0;
    if (counted) {
        a.counts = static_cast<int32_t*>(workspace);
        st = launch_dependent("expert count launch", moe_count_kernel, kMoeCountChunks, kMoeThreads, s, a.ids, a.n, a.chunk,
                              a.E, static_cast<int32_t*>(workspace));
        if (st != NVFP4LORA_OK) return st;
    }
    // a token per CTA at least, or about eight padding rows; four CTAs per SM at most
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(std::max<int64_t>(num_tokens, padded_rows / 8),
                                                                (int64_t)info->sms * 4));
    auto go = [&](auto kernel) { return launch_dependent("permute launch", kernel, grid, kMoePermuteThreads, s, a); };
    auto fits = [&](int64_t v) { return row_bytes % v == 0 && aligned(x, v) && aligned(rows, v); };
    if (fits(16)) return go(moe_permute_kernel<16>);
    if (fits(4)) return go(moe_permute_kernel<4>);
    if (fits(2)) return go(moe_permute_kernel<2>);
    return go(moe_permute_kernel<1>);
}

nvfp4lora_status nvfp4lora_moe_unpermute(const void* y, int64_t padded_rows, int64_t H, int32_t dtype,
                                         const int32_t* expanded_idx_to_permuted_idx, const float* topk_weights,
                                         int64_t num_tokens, int64_t top_k, void* out, nvfp4lora_stream stream) {
    t_last_error.clear();
    nvfp4lora_status st = check_routing(num_tokens, top_k, padded_rows);
    if (st != NVFP4LORA_OK) return st;
    if (H < 1 || H > kMaxK) return fail(NVFP4LORA_ERR_INVALID_ARG, "H = %lld: 1 <= H <= 2^20 is required", (long long)H);
    if (!valid_type(dtype)) return fail(NVFP4LORA_ERR_INVALID_ARG, "dtype must be NVFP4LORA_DTYPE_BF16, _FP16 or _FP32");
    if (num_tokens == 0) return NVFP4LORA_OK;
    if (!out || !expanded_idx_to_permuted_idx || (!y && padded_rows > 0))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "y, expanded_idx_to_permuted_idx and out must be non-null");
    const int es = type_bytes(dtype);
    if (!aligned(y, es) || !aligned(out, es) || !aligned(expanded_idx_to_permuted_idx, 4) || !aligned(topk_weights, 4))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "y and out must be aligned to their elements, the tables 4-byte aligned");
    const int64_t n = num_tokens * top_k;
    if ((st = check_apart({{"out", out, num_tokens * H * es}},
                          {{"y", y, padded_rows * H * es}, {"expanded_idx_to_permuted_idx", expanded_idx_to_permuted_idx, n * 4},
                           {"topk_weights", topk_weights, n * 4}})) != NVFP4LORA_OK)
        return st;
    int dev = 0;
    DeviceInfo* info = nullptr;
    if ((st = device_info(&dev, &info)) != NVFP4LORA_OK) return st;
    const bool vec = rows_aligned16(H * es, {y, out});
    UnpermuteArgs a;
    a.y = y;
    a.idx = expanded_idx_to_permuted_idx;
    a.w = topk_weights;
    a.out = out;
    a.H = H;
    a.segs = (int)((H + 255) / 256);
    a.units = num_tokens * a.segs;
    a.top_k = (int)top_k;
    a.rows = (int)padded_rows;
    const int64_t grid = (a.units + kMoeThreads / 32 - 1) / (kMoeThreads / 32);
    return by_type(dtype, [&](auto ty) {
        constexpr MoeType TY = decltype(ty)::value;
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        return vec ? launch_dependent("unpermute launch", moe_unpermute_kernel<TY, true>, grid, kMoeThreads, s, a)
                   : launch_dependent("unpermute launch", moe_unpermute_kernel<TY, false>, grid, kMoeThreads, s, a);
    });
}

nvfp4lora_status nvfp4lora_moe_permute_backward(const void* grad_rows, int64_t padded_rows, int64_t H, int32_t dtype,
                                                const int32_t* expanded_idx_to_permuted_idx, int64_t num_tokens,
                                                int64_t top_k, void* grad_x, nvfp4lora_stream stream) {
    // the sum of a token's rows, each with weight 1
    return nvfp4lora_moe_unpermute(grad_rows, padded_rows, H, dtype, expanded_idx_to_permuted_idx, nullptr, num_tokens,
                                   top_k, grad_x, stream);
}

nvfp4lora_status nvfp4lora_moe_unpermute_backward(const void* grad_out, const void* y, int64_t padded_rows, int64_t H,
                                                  int32_t dtype, const int32_t* expanded_idx_to_permuted_idx,
                                                  const int32_t* permuted_idx_to_expanded_idx, const int32_t* m_indptr,
                                                  int64_t num_experts, const float* topk_weights, int64_t num_tokens,
                                                  int64_t top_k, void* grad_rows, float* grad_weights,
                                                  nvfp4lora_stream stream) {
    t_last_error.clear();
    nvfp4lora_status st = check_routing(num_tokens, top_k, padded_rows);
    if (st != NVFP4LORA_OK) return st;
    if (H < 1 || H > kMaxK) return fail(NVFP4LORA_ERR_INVALID_ARG, "H = %lld: 1 <= H <= 2^20 is required", (long long)H);
    if (!valid_type(dtype)) return fail(NVFP4LORA_ERR_INVALID_ARG, "dtype must be NVFP4LORA_DTYPE_BF16, _FP16 or _FP32");
    if (num_experts < 1 || num_experts > kMoeMaxExperts)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "num_experts = %lld: 1 <= num_experts <= %d is required",
                    (long long)num_experts, kMoeMaxExperts);
    if ((topk_weights == nullptr) != (grad_weights == nullptr))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "topk_weights and grad_weights go together");
    if (!m_indptr || !aligned(m_indptr, 4))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "m_indptr must be a non-null, 4-byte aligned int32 array");
    if (num_tokens == 0 || padded_rows == 0) {
        if (num_tokens > 0)
            return fail(NVFP4LORA_ERR_INVALID_ARG, "padded_rows = 0 with num_tokens = %lld", (long long)num_tokens);
        return NVFP4LORA_OK;
    }
    if (!grad_out || !grad_rows || !expanded_idx_to_permuted_idx || !permuted_idx_to_expanded_idx || (topk_weights && !y))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "grad_out, y, grad_rows and the tables must be non-null");
    const int es = type_bytes(dtype);
    if (!aligned(grad_out, es) || !aligned(y, es) || !aligned(grad_rows, es) || !aligned(expanded_idx_to_permuted_idx, 4) ||
        !aligned(permuted_idx_to_expanded_idx, 4) || !aligned(topk_weights, 4) || !aligned(grad_weights, 4))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "rows must be aligned to their elements, the tables 4-byte aligned");
    // grad_rows may be y itself, grad_weights topk_weights: a thread reads its elements, and a block a token's weights,
    // before they are written
    const int64_t bytes = padded_rows * H * es, n = num_tokens * top_k;
    if ((st = check_apart({{"grad_rows", grad_rows, bytes}, {"grad_weights", grad_weights, n * 4}},
                          {{"grad_out", grad_out, num_tokens * H * es}, {"y", topk_weights && y != grad_rows ? y : nullptr, bytes},
                           {"expanded_idx_to_permuted_idx", expanded_idx_to_permuted_idx, n * 4},
                           {"permuted_idx_to_expanded_idx", permuted_idx_to_expanded_idx, padded_rows * 4},
                           {"m_indptr", m_indptr, (num_experts + 1) * 4},
                           {"topk_weights", topk_weights == grad_weights ? nullptr : topk_weights, n * 4}})) != NVFP4LORA_OK)
        return st;
    int dev = 0;
    DeviceInfo* info = nullptr;
    if ((st = device_info(&dev, &info)) != NVFP4LORA_OK) return st;
    const bool vec = rows_aligned16(H * es, {grad_out, y, grad_rows});
    UnpermuteBwdArgs a;
    a.g = grad_out;
    a.y = y;
    a.idx = expanded_idx_to_permuted_idx;
    a.inv = permuted_idx_to_expanded_idx;
    a.total = m_indptr + num_experts;
    a.w = topk_weights;
    a.gy = grad_rows;
    a.gw = grad_weights;
    a.H = H;
    a.T = (int)num_tokens;
    a.top_k = (int)top_k;
    a.rows = (int)padded_rows;
    const int block = (int)std::min<int64_t>(kMoeBwdThreads, (H + 255) / 256 * 32);
    // the padding rows: up to two CTAs per SM
    const int64_t grid = num_tokens + std::min<int64_t>((padded_rows + 255) / 256, 2 * (int64_t)info->sms);
    return by_type(dtype, [&](auto ty) {
        constexpr MoeType TY = decltype(ty)::value;
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        return vec ? launch_dependent("unpermute gradient launch", moe_unpermute_bwd_kernel<TY, true>, grid, block, s, a)
                   : launch_dependent("unpermute gradient launch", moe_unpermute_bwd_kernel<TY, false>, grid, block, s, a);
    });
}

nvfp4lora_status nvfp4lora_fp8_quantize(const void* x, int64_t rows, int64_t H, int32_t dtype, int64_t block_rows,
                                        uint8_t* q, float* scales, int64_t scale_stride_row, int64_t scale_stride_group,
                                        nvfp4lora_stream stream) {
    t_last_error.clear();
    nvfp4lora_status st = check_fp8_rows(x, q, scales, rows, H, dtype);
    if (st != NVFP4LORA_OK) return st;
    if (block_rows != 1 && block_rows != 128)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "block_rows = %lld: 1 or 128 is required", (long long)block_rows);
    const int64_t groups = (H + 127) / 128, brows = (rows + block_rows - 1) / block_rows;
    if ((st = check_scale_strides(brows, groups, scale_stride_row, scale_stride_group)) != NVFP4LORA_OK) return st;
    const Span sx{"x", x, rows * H * type_bytes(dtype)}, sq{"q", q, rows * H};
    if ((st = check_apart({sq}, {sx})) != NVFP4LORA_OK ||
        (st = check_apart(Scales{"scales", scales, brows, scale_stride_row, groups, scale_stride_group}, {sx, sq})) != NVFP4LORA_OK)
        return st;
    int dev = 0;
    DeviceInfo* info = nullptr;
    if ((st = device_info(&dev, &info)) != NVFP4LORA_OK) return st;
    Fp8QuantArgs a = {};
    a.x = x;
    a.q = q;
    a.scales = scales;
    a.stride_r = scale_stride_row;
    a.stride_g = scale_stride_group;
    a.rows = rows;
    a.H = H;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = H % 8 == 0 && aligned(x, 16) && aligned(q, 8);
    return by_type(dtype, [&](auto ty) {
        constexpr MoeType TY = decltype(ty)::value;
        const int64_t tiles = (rows + 127) / 128 * groups;
        if (block_rows == 128)
            return vec ? launch_dependent("quantize launch", quantize_fp8_tile_kernel<TY, true>, tiles, 256, s, a)
                       : launch_dependent("quantize launch", blocks_fp8_kernel<TY>, tiles, 256, s, a);
        return vec ? launch_dependent("quantize launch", quantize_fp8_tile_kernel<TY, false>, tiles, 256, s, a)
                   : launch_dependent("quantize launch", row_fp8_kernel<TY, false>, rows, 256, s, a);
    });
}

nvfp4lora_status nvfp4lora_rmsnorm_fp8_quantize(const void* x, void* residual, const void* weight, int64_t rows, int64_t H,
                                                int32_t dtype, float eps, void* norm_out, uint8_t* q, float* scales,
                                                int64_t scale_stride_row, int64_t scale_stride_group,
                                                nvfp4lora_stream stream) {
    t_last_error.clear();
    nvfp4lora_status st = check_fp8_rows(x, q, scales, rows, H, dtype);
    if (st != NVFP4LORA_OK) return st;
    if (!weight) return fail(NVFP4LORA_ERR_INVALID_ARG, "weight must be non-null");
    if (!(eps >= 0.0f)) return fail(NVFP4LORA_ERR_INVALID_ARG, "eps = %g: a number >= 0 is required", (double)eps);
    const int es = type_bytes(dtype);
    if (!aligned(residual, es) || !aligned(weight, es) || !aligned(norm_out, es))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "residual, weight and norm_out must be aligned to their elements");
    const int64_t groups = (H + 127) / 128;
    if ((st = check_scale_strides(rows, groups, scale_stride_row, scale_stride_group)) != NVFP4LORA_OK) return st;
    // x may be residual or norm_out itself: a thread reads its elements before it writes them
    const int64_t bytes = rows * H * es;
    const Span sx{"x", x == residual || x == norm_out ? nullptr : x, bytes}, sr{"residual", residual, bytes},
        sn{"norm_out", norm_out, bytes}, sw{"weight", weight, H * es}, sq{"q", q, rows * H};
    if ((st = check_apart({sr, sn, sq}, {sx, sw})) != NVFP4LORA_OK ||
        (st = check_apart(Scales{"scales", scales, rows, scale_stride_row, groups, scale_stride_group}, {sx, sr, sn, sw, sq})) !=
            NVFP4LORA_OK)
        return st;
    int dev = 0;
    DeviceInfo* info = nullptr;
    if ((st = device_info(&dev, &info)) != NVFP4LORA_OK) return st;
    Fp8QuantArgs a = {};
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.norm_out = norm_out;
    a.q = q;
    a.scales = scales;
    a.stride_r = scale_stride_row;
    a.stride_g = scale_stride_group;
    a.rows = rows;
    a.H = H;
    a.eps = eps;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = H % 8 == 0 && aligned(x, 16) && aligned(residual, 16) && aligned(weight, 16) &&
                     aligned(norm_out, 16) && aligned(q, 8);
    return by_type(dtype, [&](auto ty) {
        constexpr MoeType TY = decltype(ty)::value;
        // longer rows than the registers of a CTA hold are read twice
        if (H > kNormMaxThreads * 8 * 4) return launch_dependent("norm launch", row_fp8_kernel<TY, true>, rows, 256, s, a);
        // Chunks per warp: few where there are few rows, so that a row's latency is spread over many warps (16 x
        // 4096: 1.93 us with one, 2.3 with two); otherwise two, which divide once for both (8192 x 2048: 13.4 us with
        // two, 16.5 with one), and four for long rows: from 4096 on without a residual (7866 x 7168: 42 us with four,
        // 46 with two), from 8192 on with one (3000 x 8192: 31 with four, 28.7 with two).  Four chunks of element
        // accesses do not fit the registers of two CTAs.
        const bool few = rows < 8 * (int64_t)info->sms;
        if (H <= 512 && !few) {
            // a warp per row: 65536 x 512 36 us, 68 with a CTA of two warps per row
            const int64_t grid = (rows + kNormShortRows - 1) / kNormShortRows;
            if (H <= 256)
                return vec ? launch_dependent("norm launch", rmsnorm_fp8_kernel<TY, 1, true, true>, grid, 32 * kNormShortRows, s, a)
                           : launch_dependent("norm launch", rmsnorm_fp8_kernel<TY, 1, false, true>, grid, 32 * kNormShortRows, s, a);
            return vec ? launch_dependent("norm launch", rmsnorm_fp8_kernel<TY, 2, true, true>, grid, 32 * kNormShortRows, s, a)
                       : launch_dependent("norm launch", rmsnorm_fp8_kernel<TY, 2, false, true>, grid, 32 * kNormShortRows, s, a);
        }
        const int64_t one = few ? kNormMaxThreads * 8 : vec ? 768 : 2048;
        const int64_t two = few || !vec || residual ? kNormMaxThreads * 16 : 4096;
        const int per = H <= one ? 1 : H <= two ? 2 : 4;
        const int threads = (int)((H + 256 * per - 1) / (256 * per)) * 32;
        auto go = [&](auto kernel) { return launch_dependent("norm launch", kernel, rows, threads, s, a); };
        if (per == 1) return vec ? go(rmsnorm_fp8_kernel<TY, 1, true, false>) : go(rmsnorm_fp8_kernel<TY, 1, false, false>);
        if (per == 2) return vec ? go(rmsnorm_fp8_kernel<TY, 2, true, false>) : go(rmsnorm_fp8_kernel<TY, 2, false, false>);
        return vec ? go(rmsnorm_fp8_kernel<TY, 4, true, false>) : go(rmsnorm_fp8_kernel<TY, 4, false, false>);
    });
}

nvfp4lora_status nvfp4lora_mm_fp8(const uint8_t* a, const uint8_t* b, const float* a_scale, int64_t a_scale_stride_m,
                                  int64_t a_scale_stride_k, const float* b_scale, const uint16_t* bias, void* out,
                                  int32_t out_dtype, int64_t M, int64_t N, int64_t K, nvfp4lora_stream stream) {
    t_last_error.clear();
    if (M < 1) return fail(NVFP4LORA_ERR_INVALID_ARG, "M = %lld: M >= 1 is required", (long long)M);
    if (N < 1) return fail(NVFP4LORA_ERR_INVALID_ARG, "N = %lld: N >= 1 is required", (long long)N);
    if (K < 16 || K % 16 != 0)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "K = %lld: K must be a positive multiple of 16", (long long)K);
    if (M > kMaxDim || N > kMaxDim || K > kMaxK)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "M, N <= 2^30 and K <= 2^20 are required");
    if (!valid_type(out_dtype))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "out_dtype must be NVFP4LORA_DTYPE_BF16, _FP16 or _FP32");
    if (!a || !b || !a_scale || !b_scale || !out)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "a, b, a_scale, b_scale and out must be non-null");
    if (!aligned(a, 16) || !aligned(b, 16)) return fail(NVFP4LORA_ERR_INVALID_ARG, "a and b must be 16-byte aligned");
    if (!aligned(a_scale, 4) || !aligned(b_scale, 4))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "a_scale and b_scale must be 4-byte aligned");
    if (!aligned(out, type_bytes(out_dtype)) || !aligned(bias, 2))
        return fail(NVFP4LORA_ERR_INVALID_ARG, "out must be aligned to its elements and bias 2-byte aligned");
    if (a_scale_stride_m < 0 || a_scale_stride_k < 0)
        return fail(NVFP4LORA_ERR_INVALID_ARG, "a_scale strides must not be negative");
    const int64_t kblocks = (K + 127) / 128;
    const Span so{"out", out, M * N * type_bytes(out_dtype)};
    nvfp4lora_status st = check_apart({so}, {{"a", a, M * K}, {"b", b, N * K}, {"b_scale", b_scale, (N + 127) / 128 * kblocks * 4},
                                             {"bias", bias, N * 2}});
    if (st != NVFP4LORA_OK ||
        (st = check_apart(Scales{"a_scale", a_scale, M, a_scale_stride_m, kblocks, a_scale_stride_k}, {so})) != NVFP4LORA_OK)
        return st;
    int dev = 0;
    DeviceInfo* info = nullptr;
    if ((st = device_info(&dev, &info)) != NVFP4LORA_OK) return st;
    Fp8GemmArgs g = {};
    g.a_scale = a_scale;
    g.b_scale = b_scale;
    g.bias = bias;
    g.out = out;
    g.stride_am = a_scale_stride_m;
    g.stride_ak = a_scale_stride_k;
    g.M = (int)M;
    g.N = (int)N;
    g.kblocks = (int)kblocks;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (out_dtype == NVFP4LORA_DTYPE_BF16) return launch_fp8<OutType::BF16>(info, a, b, g, K, s);
    if (out_dtype == NVFP4LORA_DTYPE_FP16) return launch_fp8<OutType::FP16>(info, a, b, g, K, s);
    return launch_fp8<OutType::FP32>(info, a, b, g, K, s);
}

const char* nvfp4lora_last_error(void) { return t_last_error.c_str(); }

const char* nvfp4lora_version(void) { return "nvfp4lora 0.1.0 (sm_100a)"; }

}  // extern "C"
