// Bounded waits of the attention kernels, launched by test_attention_waits.py.
//
// dkdv_behind: dK and dV of the bf16 backward pass behind a slow kernel.  The library launches
// attn_dkdv_tc_kernel beside the last blocks of the kernel that forms delta; here that one
// is replaced by a kernel that lets its successor start at once, takes as long as it is
// told and only then writes delta.
// run_out: a wait on a barrier that nothing arrives at.
#include "lard_host.h"
#include "attn/attn_bwd_tc.cuh"

using namespace lard::attn;
using bf16 = __nv_bfloat16;

__global__ void slow_delta(const float* from, float* delta, int rows, unsigned long long ns) {
    next_may_start();
    const uint64_t t0 = lard::ptx::globaltimer_ns();
    for (int k = 0; k < (1 << 20) && lard::ptx::globaltimer_ns() - t0 < ns; ++k) __nanosleep(1000);
    for (int r = threadIdx.x; r < rows; r += blockDim.x) delta[r] = from[r];
}

// Contiguous [heads, rows, d].
static bool map_of(EncodeTiledFn encode, CUtensorMap* m, const void* p, int heads, int rows, int d, unsigned box) {
    const cuuint64_t line = 2ull * d;
    cuuint64_t dims[4] = {cuuint64_t(d), cuuint64_t(rows), cuuint64_t(heads), 1};
    cuuint64_t strides[3] = {line, line * rows, line * rows * heads};
    cuuint32_t boxes[4] = {64, box, 1, 1}, steps[4] = {1, 1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dims, strides, boxes, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
static int run(bf16* q, bf16* k, bf16* v, bf16* dout, bf16* dk, bf16* dv, float* lse, float* from, float* delta, int Hq,
               int Hkv, int n, int m, float tau, unsigned before_us, unsigned wait_us) {
    const EncodeTiledFn encode = find_encode_tiled();
    TcBwdArgs g = {};
    if (!encode || !map_of(encode, &g.k, k, Hkv, m, D, 128) || !map_of(encode, &g.v, v, Hkv, m, D, 128) ||
        !map_of(encode, &g.q64, q, Hq, n, D, kUnit) || !map_of(encode, &g.do64, dout, Hq, n, D, kUnit))
        return -1;
    g.dk = View<bf16>{dk, 0, static_cast<long long>(m) * D, D};
    g.dv = View<bf16>{dv, 0, static_cast<long long>(m) * D, D};
    g.lse = lse;
    g.delta = delta;
    g.m = m;
    g.B = 1;
    g.Hkv = Hkv;
    g.G = Hq / Hkv;
    g.n = n;
    g.qsplits = g.ksplits = 1;
    g.khead = g.vhead = g.qhead = g.dohead = 1;
    g.cfac = tau * kLog2e;
    g.tau = tau;
    g.wait_ns = 1000ull * wait_us;
    g.drain_ns = 1000000000ull;
    if (set_smem(attn_dkdv_tc_kernel<D>, DkvLayout<D>::SMEM_BYTES) != cudaSuccess ||
        !split_fits(attn_dkdv_tc_kernel<D>, kBwdTcThreads, kDqRegsSplitTotal))
        return -2;
    slow_delta<<<1, 256>>>(from, delta, Hq * n, 1000ull * before_us);
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((m + 127) / 128 * Hkv);
    c.blockDim = dim3(kBwdTcThreads);
    c.dynamicSmemBytes = DkvLayout<D>::SMEM_BYTES;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    if (cudaLaunchKernelEx(&c, attn_dkdv_tc_kernel<D>, g) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return -3;
    unsigned int fault = 0;
    if (cudaMemcpyFromSymbol(&fault, lard::g_lard_fault, sizeof(fault)) != cudaSuccess) return -4;
    return static_cast<int>(fault);
}

// On the current device's default stream.  Returns the fault bits, or a negative number if a
// call failed.
extern "C" __attribute__((visibility("default"))) int dkdv_behind(int d, void* q, void* k, void* v, void* dout, void* dk, void* dv, void* lse, void* from,
                           void* delta, int Hq, int Hkv, int n, int m, float tau, unsigned before_us, unsigned wait_us) {
    auto h = [](void* p) { return static_cast<bf16*>(p); };
    auto f = [](void* p) { return static_cast<float*>(p); };
    return (d == 64 ? run<64> : run<128>)(h(q), h(k), h(v), h(dout), h(dk), h(dv), f(lse), f(from), f(delta), Hq, Hkv, n, m,
                                          tau, before_us, wait_us);
}

// What bounded waits do: got[0..3] = whether the wait returned true, microseconds that it took,
// twice (an mbarrier that nothing arrives at; the same when the block has given up);
// got[4] = an mbarrier whose phase is complete.  Then the exit wait runs out.
__global__ void waits_run_out(unsigned long long ns, unsigned int* got) {
    __shared__ uint64_t bar[2];
    __shared__ int abort_flag;
    if (threadIdx.x != 0) return;
    abort_flag = 0;
    lard::ptx::mbar_init(&bar[0], 1);
    lard::ptx::mbar_init(&bar[1], 1);
    lard::ptx::fence_mbar_init();
    lard::ptx::mbar_arrive(&bar[1]);
    for (int k = 0; k < 2; ++k) {
        const uint64_t t0 = lard::ptx::globaltimer_ns();
        got[2 * k] = mbar_wait(&bar[0], 0, &abort_flag, k ? 1000 * ns : ns, &lard::g_lard_fault, lard::kFaultBwdMma);
        got[2 * k + 1] = static_cast<unsigned int>((lard::ptx::globaltimer_ns() - t0) / 1000);
    }
    got[4] = mbar_wait(&bar[1], 0, &abort_flag, ns, &lard::g_lard_fault, lard::kFaultBwdProducer);
    lard::drain(&bar[0], 0, ns);
}

// Returns the fault bits, which it clears, or a negative number if a call failed.
extern "C" __attribute__((visibility("default"))) int run_out(unsigned limit_us, unsigned int* got) {
    waits_run_out<<<1, 32>>>(1000ull * limit_us, got);
    if (cudaDeviceSynchronize() != cudaSuccess) return -1;
    unsigned int fault = 0;
    const unsigned int zero = 0;
    if (cudaMemcpyFromSymbol(&fault, lard::g_lard_fault, sizeof(fault)) != cudaSuccess ||
        cudaMemcpyToSymbol(lard::g_lard_fault, &zero, sizeof(zero)) != cudaSuccess)
        return -2;
    return static_cast<int>(fault);
}
