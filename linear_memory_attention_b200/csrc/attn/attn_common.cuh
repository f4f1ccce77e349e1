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
    View<T> out, rest;  // rest: what rounding left of out, or p = NULL
    float* lse;         // [B, Hq, n]
    KeySeg<T> seg[2];
    int nseg;
    int PB, Hkv, G, n, R;
    float cfac;  // tau * log2(e): logit -> log2 domain
    // With join, the key tiles of a problem are dealt to `splits` blocks, each of
    // which leaves its rows' normalised O and LSE as partials split0 + split.
    int splits, split0, join;
    int second;       // the call's second pass, which runs beside the first
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

// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void copy16_or_0(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The pointer that lane `from` holds.
template <typename T>
__device__ __forceinline__ T* shfl_ptr(T* p, int from) {
    return reinterpret_cast<T*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), from));
}

// A warp brings rows [first, last) of its 32 rows of D bf16 to shared memory, as
// K-major operand rows (64-column chunks 16 KB apart, 128-byte rows, 128-byte
// swizzle) from row0 on.  Lane r holds row r's address, or NULL for zeros.
// Neighbouring lanes read neighbouring pieces of a row: one row a lane would
// touch 32 rows with every instruction.
template <int D>
__device__ __forceinline__ void rows_to_operand(uint32_t tile, int row0, const __nv_bfloat16* mine, int lane, int first,
                                                int last) {
    constexpr int kLanes = D / 8;  // lanes of a row
#pragma unroll 4
    for (int k = first; k < last; k += 32 / kLanes) {
        const int r = k + lane / kLanes, u = lane % kLanes;
        const __nv_bfloat16* src = shfl_ptr(mine, r);
        const int row = row0 + r;
        copy16_or_0(tile + (u >> 3) * 16384 + row * 128 + (((u & 7) ^ (row & 7)) << 4), src ? src + u * 8 : nullptr, src);
    }
}

// A warp writes its 32 rows of ROW bytes from a staging area of its own (32 ROW
// bytes of shared memory) to global memory.  Lane r has put row r's 16-byte
// units at stage_unit(r, u) and holds its address, or NULL to skip it.
template <int ROW>
__device__ __forceinline__ uint32_t stage_unit(uint32_t stage, int r, int u) {
    // Eight lanes in a row (rows when writing, units when reading) use different banks.
    return stage + r * ROW + ((u ^ (ROW >= 128 ? r & 7 : r >> 1 & 3)) << 4);
}
template <int ROW>
__device__ __forceinline__ void staged_rows_out(uint32_t stage, void* mine, int lane) {
    constexpr int kLanes = ROW / 16;  // lanes of a row
    __syncwarp();
#pragma unroll 4
    for (int k = 0; k < 32; k += 32 / kLanes) {
        const int r = k + lane / kLanes, u = lane % kLanes;
        char* dst = shfl_ptr(static_cast<char*>(mine), r);
        uint4 x;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "r"(stage_unit<ROW>(stage, r, u))
                     : "memory");
        if (dst) *reinterpret_cast<uint4*>(dst + u * 16) = x;
    }
    __syncwarp();  // the area may be written again
}

// Rounds 32 fp32 columns, times `scale`, to bf16 into units first and up of a staged row of ROW bytes.
template <int ROW>
__device__ __forceinline__ void stage_bf16(uint32_t area, int lane, int first, const float (&o)[32], float scale) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
        ptx::st_shared_v4(stage_unit<ROW>(area, lane, first + u), ptx::pack_bf16x2(o[8 * u] * scale, o[8 * u + 1] * scale),
                          ptx::pack_bf16x2(o[8 * u + 2] * scale, o[8 * u + 3] * scale),
                          ptx::pack_bf16x2(o[8 * u + 4] * scale, o[8 * u + 5] * scale),
                          ptx::pack_bf16x2(o[8 * u + 6] * scale, o[8 * u + 7] * scale));
}

// What rounding to bf16 leaves of x.
__device__ __forceinline__ float rounding_rest(float x) { return x - __bfloat162float(__float2bfloat16_rn(x)); }

// The same of 32 values, in pairs (a conversion of two costs what one of one does).
__device__ __forceinline__ void leave_rest(float (&o)[32]) {
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
        const uint32_t w = ptx::pack_bf16x2(o[k], o[k + 1]);
        o[k] -= __uint_as_float(w << 16);
        o[k + 1] -= __uint_as_float(w & 0xffff0000u);
    }
}

// Writes 32 fp32 columns of a warp's 32 rows, COLS at a time through the area.
template <int COLS>
__device__ __forceinline__ void fp32_rows_out(uint32_t area, int lane, const float (&o)[32], float* mine) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(o);
#pragma unroll
    for (int x = 0; x < 32; x += COLS) {
#pragma unroll
        for (int u = 0; u < COLS / 4; ++u)
            ptx::st_shared_v4(stage_unit<COLS * 4>(area, lane, u), w[x + 4 * u], w[x + 4 * u + 1], w[x + 4 * u + 2],
                              w[x + 4 * u + 3]);
        staged_rows_out<COLS * 4>(area, mine ? mine + x : nullptr, lane);
    }
}

}  // namespace attn
}  // namespace lard
