// attn_ptx.cuh -- the sm_100a instructions that the attention kernels use
// beside those of sm100_ptx.cuh.
#pragma once

#include "../sm100_ptx.cuh"

namespace lard {
namespace attn {

// Programmatic dependent launch: the next kernel of the call may start as soon
// as every block of this one has begun (its blocks then fill SMs that this one
// leaves idle); whoever reads what the kernel before wrote waits first.
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(ptx::smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// ptx::mbar_wait with the clock and the abort flag looked at once in 64 tries:
// reading %globaltimer takes hundreds of cycles, by which each wait that does
// not find its phase complete at once would be late.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns,
                                          unsigned int* fault_word, unsigned int code) {
    for (int k = 0; k < 64; ++k)
        if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    while (true) {
        for (int k = 0; k < 64; ++k)
            if (ptx::mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (ptx::globaltimer_ns() - t0 > limit_ns) {
            *abort_flag = 1;
            atomicOr(fault_word, code);
            return false;
        }
    }
}

// umma_ts with the accumulate flag at run time.
__device__ __forceinline__ void umma_ts_acc(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 db, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(accumulate), "r"(idesc)
        : "memory");
}

}  // namespace attn
}  // namespace lard
