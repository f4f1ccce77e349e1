// attn_join.cuh -- what is left when an axis was split over blocks: joining the
// forward pass's partial rows, adding the backward pass's partial sums.
// Both read what the blocks before left in L2 and are bound by that.
#pragma once

#include "attn_common.cuh"
#include "attn_ptx.cuh"

namespace lard {
namespace attn {

// Joins the splits of a row: LSE = log sum_s exp LSE_s, O = sum_s exp(LSE_s - LSE) O_s.
// One warp per row; lanes share the splits' weights, then the head dimension.
template <typename T, int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ FwdArgs<T> g) {
    wait_for_kernel_before();
    const int lane = threadIdx.x & 31;
    const long long row = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (row >= g.rows) return;
    constexpr int E = D / 32;
    float top = -INFINITY;
    for (int s = lane; s < g.splits; s += 32) top = fmaxf(top, g.part_lse[s * g.rows + row]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float base = top == -INFINITY ? 0.f : top;
    float total = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int s0 = 0; s0 < g.splits; s0 += 32) {
        const int here = min(32, g.splits - s0);
        const float mine = lane < here ? exp2f((g.part_lse[(s0 + lane) * g.rows + row] - base) * kLog2e) : 0.f;
#pragma unroll 8
        for (int s = 0; s < here; ++s) {
            const float w = __shfl_sync(0xffffffffu, mine, s);
            total += w;
            // A split that saw nothing need not have written its O.
            const float* src = g.part_o + ((w == 0.f ? 0 : s0 + s) * g.rows + row) * D + lane * E;
            float x[E];
            if constexpr (E == 4) {
                const float4 v = load4(src);
                x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
            } else {
                const float2 v = *reinterpret_cast<const float2*>(src);
                x[0] = v.x; x[1] = v.y;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = w == 0.f ? o[e] : fmaf(w, x[e], o[e]);
        }
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const int R = g.G * g.n;
    const int bh = static_cast<int>(row / R), r = static_cast<int>(row % R);
    T* dst = g.out.row(bh / g.Hkv, bh % g.Hkv * g.G + r / g.n, r % g.n) + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = static_cast<T>(o[e] * inv);
    if (g.rest.p) {
        T* rest = g.rest.row(bh / g.Hkv, bh % g.Hkv * g.G + r / g.n, r % g.n) + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) rest[e] = static_cast<T>(o[e] * inv - static_cast<float>(dst[e]));
    }
    if (lane == 0) g.lse[row] = total == 0.f ? -INFINITY : base + log2f(total) * kLn2;
}

// Sums of up to three gradients: dst row = scale * sum_s src[s][row], s in order.
template <typename T>
struct SumArgs {
    struct Job {
        const float* src;
        View<T> dst;
        int splits, heads, per_head;  // rows (b, head, i)
        long long rows;
        float scale;
    } job[3];
    int jobs;
};

// One warp per row; grid over the jobs' rows one after the other.
template <typename T, int D>
__global__ void __launch_bounds__(256) attn_sum_kernel(const __grid_constant__ SumArgs<T> g) {
    wait_for_kernel_before();
    const int lane = threadIdx.x & 31;
    long long row = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    int k = 0;
    while (k < g.jobs && row >= g.job[k].rows) row -= g.job[k++].rows;
    if (k == g.jobs) return;
    const typename SumArgs<T>::Job& j = g.job[k];
    constexpr int E = D / 32;
    float o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int s = 0; s < j.splits; ++s) {
        const float* src = j.src + (s * j.rows + row) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += src[e];
    }
    const int bh = static_cast<int>(row / j.per_head), i = static_cast<int>(row % j.per_head);
    T* dst = j.dst.row(bh / j.heads, bh % j.heads, i) + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = static_cast<T>(o[e] * j.scale);
}

}  // namespace attn
}  // namespace lard
