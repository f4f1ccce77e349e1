// attn_join.cuh -- what is left when an axis was split over blocks: joining the
// forward pass's partial rows, adding the backward pass's partial sums.
// Both read what the blocks before left in L2 or HBM and are bound by that (131072 rows
// of two parts at d = 128: 168 MB in and out in 52 us with the launch).
#pragma once

#include <type_traits>

#include "attn_common.cuh"
#include "attn_ptx.cuh"

namespace lard {
namespace attn {

// E (2 or 4) values that a lane reads or writes in one piece.
template <int E>
__device__ __forceinline__ void load_piece(const float* p, float (&x)[E]) {
    if constexpr (E == 4) {
        const float4 v = load4(p);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
        const float2 v = *reinterpret_cast<const float2*>(p);
        x[0] = v.x; x[1] = v.y;
    }
}
template <int E>
__device__ __forceinline__ void store_piece(float* p, const float (&x)[E]) {
    if constexpr (E == 4) store4(p, make_float4(x[0], x[1], x[2], x[3]));
    else *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
}
template <int E>
__device__ __forceinline__ void store_piece(__nv_bfloat16* p, const float (&x)[E]) {
    if constexpr (E == 4) store4(p, make_float4(x[0], x[1], x[2], x[3]));
    else *reinterpret_cast<uint32_t*>(p) = ptx::pack_bf16x2(x[0], x[1]);
}

// Joins the splits of a row: LSE = log sum_s exp LSE_s, O = sum_s exp(LSE_s - LSE) O_s.
// One warp per row; lanes share the splits' weights, then the head dimension.  The
// parts of four splits are requested at a time, the first before the weights are known.
template <typename T, int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ FwdArgs<T> g) {
    wait_for_kernel_before();
    const int lane = threadIdx.x & 31;
    const long long row = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (row >= g.rows) return;
    constexpr int E = D / 32, kBatch = 4;
    const float* part = g.part_o + row * D + lane * E;
    float x[kBatch][E];
    auto request = [&](int s) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (s + k < g.splits) load_piece<E>(part + (s + k) * g.rows * D, x[k]);
    };
    request(0);
    float top = -INFINITY;
    for (int s = lane; s < g.splits; s += 32) top = fmaxf(top, g.part_lse[s * g.rows + row]);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
    const float base = top == -INFINITY ? 0.f : top;
    float total = 0.f, o[E], mine = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int s = 0; s < g.splits; s += kBatch) {
        if (s > 0) request(s);
        if (s % 32 == 0) mine = s + lane < g.splits ? exp2f((g.part_lse[(s + lane) * g.rows + row] - base) * kLog2e) : 0.f;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const float w = __shfl_sync(0xffffffffu, mine, (s + k) % 32);
            if (s + k >= g.splits) continue;
            total += w;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = w == 0.f ? o[e] : fmaf(w, x[k][e], o[e]);
        }
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const int R = g.G * g.n;
    const int bh = static_cast<int>(row / R), r = static_cast<int>(row % R);
    const int b = bh / g.Hkv, head = bh % g.Hkv * g.G + r / g.n, pos = r % g.n;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= inv;
    store_piece<E>(g.out.row(b, head, pos) + lane * E, o);
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        if (g.rest.p) {
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = rounding_rest(o[e]);
            store_piece<E>(g.rest.row(b, head, pos) + lane * E, o);
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
#pragma unroll 2
    for (int s = 0; s < j.splits; ++s) {
        float x[E];
        load_piece<E>(j.src + (s * j.rows + row) * D + lane * E, x);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += x[e];
    }
    const int bh = static_cast<int>(row / j.per_head), i = static_cast<int>(row % j.per_head);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= j.scale;
    store_piece<E>(j.dst.row(bh / j.heads, bh % j.heads, i) + lane * E, o);
}

}  // namespace attn
}  // namespace lard
