// What the products over 8-bit floating-point operands share: waits, the MMA,
// cluster barriers.  sm_103a only.
#pragma once

#include "q2k_common.cuh"
#include "q2k_umma.cuh"

namespace q2k {

// mbar_wait_bounded with its clock read only after many polls: here most
// waits are short, and each lies on the path from one block of K to the next.
__device__ __forceinline__ bool mbar_wait_near(uint32_t bar, uint32_t parity, const volatile int* abort_flag)
{
    uint64_t t0 = 0;
    for (uint32_t it = 0;; ++it) {
        if (mbar_try_wait(bar, parity))
            return true;
        if ((it & 63u) == 63u) {
            if (*abort_flag)
                return false;
            const uint64_t t = global_timer_ns();
            if (t0 == 0)
                t0 = t;
            else if (t - t0 > 2000000000ull)
                return false;
        }
    }
}

// A wait on a barrier whose phase has long completed still takes 85 to 120
// cycles, so the loops below ask for the next stage's barriers before they
// work on this one's, and wait only where the answer was no.  By a whole warp.
__device__ __forceinline__ bool mbar_ready(uint32_t bar, uint32_t parity) { return mbar_test_wait(bar, parity); }

// The same value in every lane, known to the compiler as such: operands of an
// MMA that are computed from it need no moves to uniform registers.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// The shared memory to launch with: all but 8 KB of what a block may have.  These kernels take all of tensor memory, and
// a block that finds it taken waits until it is given back.  Two clusters that each had one block waiting for the
// other's would wait for ever, as would a block whose tensor memory is held by a launch that waits for it; so no second
// block that works in tensor memory (none does with less than 8 KB for its operands) may fit on an SM beside one of these.
inline size_t alone_on_sm(size_t bytes, size_t most)
{
    const size_t least = most - 8192;
    return bytes < least ? least : bytes;
}

// The low and high word of smem_desc_sw128(), the address in the low one.
__device__ __forceinline__ uint64_t desc_at(uint32_t addr)
{
    constexpr uint32_t kHi = (1024u >> 4) | 1u << 14 | 2u << 29;
    return (uint64_t)kHi << 32 | (1u << 16 | (addr >> 4));
}

// Instruction descriptor: D fp32, A and B e4m3, both K-major, M = 128.
constexpr uint32_t instr_desc_e4m3(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24); }
constexpr uint32_t kBIsE5m2 = 1u << 10;  // (each operand of kind::f8f6f4 has a type of its own)

__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}

// Waits for this warp's loads from tensor memory; what uses the values comes after.
template <int N>
__device__ __forceinline__ void settle(float (&v)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; i += 8)
        asm volatile(""
                     : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]),
                       "+f"(v[i + 6]), "+f"(v[i + 7]));
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ void cluster_sync()
{
    cluster_arrive();
    cluster_wait();
}

}  // namespace q2k
