// drain_ring of the library's ring helpers against copies that land late, or never: one CTA, thread 0 arms a ring's
// barriers as a producer does, thread 32 plays the copies.
#include <cstdint>

#include "ptx.cuh"

using namespace nvfp4lora;

namespace {

constexpr uint32_t kMaxStages = 8, kBytes = 512;

// Takes bytes off the barrier's phase, as a copy that lands.
__device__ void land(uint64_t* bar) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(kBytes) : "memory");
}

__device__ void pause_ns(unsigned long long ns) {
    const unsigned long long t0 = global_timer_ns();
    while (global_timer_ns() - t0 < ns) {}
}

// out: {items landed when the drain returned, the time it took in us}
__global__ void ring_drain_kernel(uint32_t stages, uint32_t n, uint32_t missing, unsigned long long delay_ns,
                                  unsigned long long limit_ns, uint32_t* out) {
    __shared__ __align__(8) uint64_t full[kMaxStages];
    __shared__ volatile uint32_t landed;
    const uint32_t first = n > stages ? n - stages : 0;
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < stages; ++s) mbar_init(&full[s], 1);
        fence_mbar_init();
        landed = 0;
        for (uint32_t k = 0; k < n; ++k) {
            mbar_arrive_expect_tx(&full[k % stages], kBytes);
            if (k < first) land(&full[k % stages]);              // consumed long ago
        }
    }
    __syncthreads();
    if (threadIdx.x == 32) {
        for (uint32_t k = n; k-- > first;) {                     // the last one first
            pause_ns(delay_ns);
            if (k == missing) continue;
            landed = landed + 1;
            __threadfence_block();
            land(&full[k % stages]);
        }
    } else if (threadIdx.x == 0) {
        const unsigned long long t0 = global_timer_ns();
        drain_ring(full, stages, n, limit_ns);
        out[1] = (uint32_t)((global_timer_ns() - t0) / 1000);
        out[0] = landed;
    }
    __syncthreads();
}

}  // namespace

// missing: an item that never lands, or n for none.  0, or a CUDA error.
extern "C" int ring_drain(uint32_t stages, uint32_t n, uint32_t missing, uint64_t delay_ns, uint64_t limit_ns, uint32_t* out) {
    if (stages < 1 || stages > kMaxStages || n > 1000 || delay_ns > 1000000 || limit_ns > 100000000) return -1;
    uint32_t* d = nullptr;
    cudaError_t e = cudaMalloc(&d, 8);
    if (e != cudaSuccess) return (int)e;
    ring_drain_kernel<<<1, 64>>>(stages, n, missing, delay_ns, limit_ns, d);
    e = cudaMemcpy(out, d, 8, cudaMemcpyDeviceToHost);
    cudaFree(d);
    return (int)e;
}
