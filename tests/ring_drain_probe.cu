// ring_drain (csrc/w8a16_device.cuh) by itself: a warp asks for steps 0 .. steps - 1 of 8 KB by bulk
// copies into a ring of three slots, takes the first `taken` as the kernels do, and then, with up to three copies on
// their way as after a wait that gave up, drains the ring and reads what the slots hold.
#include <cuda_runtime.h>

#include "w8a16_device.cuh"

using namespace w8a16;

constexpr unsigned kStages = 3, kBytes = 8192;

__device__ DeviceStatus g_status;

__global__ void probe(const uint8_t* src, unsigned taken, unsigned steps, uint8_t* out) {
    __shared__ __align__(128) uint8_t ring[kStages][kBytes];
    __shared__ uint64_t full[kStages];
    __shared__ int abort_flag;
    const unsigned lane = threadIdx.x;
    if (lane == 0) {
        for (unsigned i = 0; i < kStages; ++i) mbar_init(smem_u32(&full[i]), 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncwarp();
    const auto issue = [&](unsigned q) {
        if (q >= steps || lane != 0) return;
        const uint32_t bar = smem_u32(&full[q % kStages]);
        mbar_arrive_expect_tx(bar, kBytes);
        asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(ring[q % kStages])),
                     "l"(src + static_cast<size_t>(q) * kBytes), "r"(kBytes), "r"(bar)
                     : "memory");
    };
    for (unsigned q = 0; q < kStages; ++q) issue(q);
    for (unsigned q = 0; q < taken; ++q) {
        mbar_wait_for(smem_u32(&full[q % kStages]), (q / kStages) & 1, 1000000000ull, &abort_flag, &g_status, 1);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        issue(q + kStages);
    }
    abort_flag = 1;
    const unsigned end = min(taken + kStages, steps);
    ring_drain<kStages>(full, taken, end, 1000000000ull, &g_status, 2);
    for (unsigned q = taken; q < end; ++q)
        for (unsigned i = lane; i < kBytes; i += 32) out[(q - taken) * kBytes + i] = ring[q % kStages][i];
}

// A slot that no copy was asked for: the drain ends at its limit and says so.
__global__ void probe_limit(unsigned long long limit_ns) {
    __shared__ uint64_t full[kStages];
    if (threadIdx.x == 0) {
        for (unsigned i = 0; i < kStages; ++i) mbar_init(smem_u32(&full[i]), 1);
        fence_barrier_init();
    }
    __syncwarp();
    ring_drain<kStages>(full, 0, 2, limit_ns, &g_status, 7);
}

extern "C" __attribute__((visibility("default"))) int ring_drain_probe(const void* src, unsigned taken, unsigned steps, void* out) {
    probe<<<1, 32>>>(static_cast<const uint8_t*>(src), taken, steps, static_cast<uint8_t*>(out));
    return static_cast<int>(cudaDeviceSynchronize());
}
extern "C" __attribute__((visibility("default"))) int ring_drain_limit(unsigned long long limit_ns) {
    probe_limit<<<1, 32>>>(limit_ns);
    return static_cast<int>(cudaDeviceSynchronize());
}
extern "C" __attribute__((visibility("default"))) int ring_drain_status(unsigned* words) {
    return static_cast<int>(cudaMemcpyFromSymbol(words, g_status, sizeof(DeviceStatus)));
}
