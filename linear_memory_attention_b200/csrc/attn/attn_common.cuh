// attn_common.cuh -- what the attention kernels share: tensor views, key
// segments, element conversion and the row arithmetic of grouped heads.
#pragma once

#include <cuda_bf16.h>

#include <climits>
#include <cstdint>

#include "../lard_kernel_common.cuh"

namespace lard {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Element (b, h, i, c) at p + b * sb + h * sh + i * sn + c (strides in elements).
template <typename T>
struct View {
    T* p;
    long long sb, sh, sn;
    __device__ __forceinline__ T* row(int b, int h, int i) const { return p + b * sb + h * sh + i * sn; }
};

// A run of keys: the rows [0, length of sequence b) of one K and one V tensor.
// causal: row i of the n newest rows sees the keys j <= length - n + i only.
template <typename T>
struct KeySeg {
    View<const T> k, v;
    const int* len;  // per sequence, or NULL: cap rows
    int cap;         // rows in memory
    int causal;
    __device__ __forceinline__ int length(int b) const {
        if (!len) return cap;
        const int l = len[b];
        return l < 0 ? 0 : (l > cap ? cap : l);
    }
};

// Forward work over one or two key segments, one after the other: PB problems
// per key head, of R query rows each; row r of problem pb is sequence
// b = pb + r / (G n), query head hk G + r % (G n) / n, row r % n.
// (Keys of their own: PB = B, R = G n.  Shared keys: PB = 1, R = B G n.)
template <typename T>
struct FwdArgs {
    View<const T> q;
    View<T> out;
    float* lse;  // [B, Hq, n]
    KeySeg<T> seg[2];
    int nseg;
    int PB, Hkv, G, n, R;
    float cfac;  // tau * log2(e): logit -> log2 domain
    // With join, the key tiles of a problem are dealt to `splits` blocks, each of
    // which leaves its rows' normalised O and LSE as partials split0 + split.
    int splits, split0, join;
    long long rows;   // B Hkv G n
    float* part_o;    // [partials][rows][D]
    float* part_lse;  // [partials][rows]
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(ptx::pack_bf16x2(v.x, v.y), ptx::pack_bf16x2(v.z, v.w));
}

// Keys of a causal segment of length len that row i of n sees: [0, limit).
__device__ __forceinline__ int causal_limit(int len, int n, int i) {
    const long long e = static_cast<long long>(len) - n + i + 1;
    return e < 0 ? 0 : (e > len ? len : static_cast<int>(e));
}

}  // namespace attn
}  // namespace lard
