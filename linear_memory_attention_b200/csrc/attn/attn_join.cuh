// attn_join.cuh -- what is left when an axis was split over blocks: joining the
// forward pass's partial rows, adding the backward pass's partial sums.
// Both read what the blocks before left in L2 or HBM and are bound by that (131072 rows
// of two parts at d = 128: 168 MB in and out in 47 us, while HBM also takes what L2 could
// not keep of the parts).
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

// First row of a warp of a join: 256 threads a block, rpw rows a warp.  The number of a thread in
// the grid would pass 32 bits from 2^30 rows on.
constexpr int kJoinThreads = 256;
__host__ __device__ constexpr unsigned join_row(unsigned block, unsigned thread, unsigned rpw) {
    return (block * (kJoinThreads / 32) + thread / 32) * rpw;
}
static_assert(join_row(0, 95, 8) == 16 && join_row(2, 32, 1) == 17, "rows of the first warps");
static_assert(join_row((1u << 24) - 1, 255, 8) == (1u << 30) - 8 && join_row(1u << 24, 0, 8) == 1u << 30 &&
                  join_row((0x7fffffffu - 1) / 64, 255, 8) == 0x7ffffff8u,
              "rows of the last warps");

// Joins the splits of a row: LSE = log sum_s exp LSE_s, O = sum_s exp(LSE_s - LSE) O_s.
// A warp has RPW rows (1 or 8): its lanes share the rows' weights, LPR lanes a row, then
// row by row the head dimension, with the parts of four splits requested at a time.
// What a row costs beside its bytes (weights, divisions for its address) is then done
// for eight rows at once: 131072 rows of two parts take 54 us with one row a warp, 47 us
// with eight.  Few rows are left to a warp each, and the first parts are requested
// before the weights are known.
template <typename T, int D, int RPW>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ FwdArgs<T> g) {
    wait_for_kernel_before();
    constexpr int E = D / 32, LPR = 32 / RPW, kBatch = 4;
    const int lane = threadIdx.x & 31, sub = lane % LPR;
    const unsigned rows = static_cast<unsigned>(g.rows);  // below 2^31 where there is a join
    const unsigned row0 = join_row(blockIdx.x, threadIdx.x, RPW), row = row0 + lane / LPR;
    if (row0 >= rows) return;
    const bool in = row < rows;
    const float* part = g.part_o + static_cast<size_t>(row0) * D + lane * E;
    auto request = [&](float (&x)[kBatch][E], int k, int s) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (s + j < g.splits && row0 + k < rows) load_piece<E>(part + ((s + j) * g.rows + k) * D, x[j]);
    };
    float first[kBatch][E];
    if (RPW == 1) request(first, 0, 0);
    auto lse_of = [&](int s) { return in && s < g.splits ? g.part_lse[s * g.rows + row] : -INFINITY; };
    float top = -INFINITY, total = 0.f;
    for (int s = sub; s < g.splits; s += LPR) top = fmaxf(top, lse_of(s));
#pragma unroll
    for (int k = LPR / 2; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
    const float base = top == -INFINITY ? 0.f : top;
    for (int s = sub; s < g.splits; s += LPR) total += exp2f((lse_of(s) - base) * kLog2e);
#pragma unroll
    for (int k = LPR / 2; k > 0; k >>= 1) total += __shfl_xor_sync(0xffffffffu, total, k);
    const float inv = total == 0.f ? 0.f : 1.f / total;

    float o[RPW][E];
#pragma unroll
    for (int k = 0; k < RPW; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) o[k][e] = 0.f;
    for (int s0 = 0; s0 < g.splits; s0 += LPR) {
        const float mine = exp2f((lse_of(s0 + sub) - base) * kLog2e) * inv;
        for (int j0 = 0; j0 < LPR && s0 + j0 < g.splits; j0 += kBatch) {
#pragma unroll
            for (int k = 0; k < RPW; ++k) {
                float x[kBatch][E];
                if (RPW > 1 || s0 + j0 > 0) request(x, k, s0 + j0);
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const float w = __shfl_sync(0xffffffffu, mine, k * LPR + j0 + j);
                    if (w == 0.f) continue;  // nothing seen, or no such split
#pragma unroll
                    for (int e = 0; e < E; ++e) o[k][e] = fmaf(w, RPW == 1 && s0 + j0 == 0 ? first[j][e] : x[j][e], o[k][e]);
                }
            }
        }
    }
    const unsigned R = static_cast<unsigned>(g.G) * g.n, at = in ? row : 0;
    const int bh = static_cast<int>(at / R), r = static_cast<int>(at % R);
    const int b = bh / g.Hkv, head = bh % g.Hkv * g.G + r / g.n, pos = r % g.n;
    T* out = g.out.row(b, head, pos);
    T* rest = g.rest.p ? g.rest.row(b, head, pos) : nullptr;
#pragma unroll
    for (int k = 0; k < RPW; ++k) {
        T* dst = shfl_ptr(out, k * LPR);
        if (row0 + k < rows) store_piece<E>(dst + lane * E, o[k]);
        if constexpr (std::is_same<T, __nv_bfloat16>::value)
            if (g.rest.p) {
                dst = shfl_ptr(rest, k * LPR);
#pragma unroll
                for (int e = 0; e < E; ++e) o[k][e] = rounding_rest(o[k][e]);
                if (row0 + k < rows) store_piece<E>(dst + lane * E, o[k]);
            }
    }
    if (in && sub == 0) g.lse[row] = total == 0.f ? -INFINITY : base + log2f(total) * kLn2;
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
