// attn_simt.cuh -- attention of fp32 tensors, on the CUDA cores.
//
// The tensor cores would round fp32 operands, so the products run on the FMA
// pipe, which bounds them (128 multiply-adds a cycle and SM).  A block of 128
// threads works on 64 x 64 tiles (16 x 64 where there are few rows): a
// thread owns 8 x 4 logits, which takes half of the shared-memory bandwidth that
// 4 x 4 takes, and tiles arrive by cp.async a step ahead, since only four warps
// share an SM at d = 128.  Multiply-adds are packed in pairs.
// Forward: running row maximum and sum in the log2 domain, P through shared
// memory, O in registers.  Backward: one kernel for each side of the logits, so that every
// sum has one owner and a fixed order (no atomics): dQ by blocks of 64 rows
// over the keys (it also forms delta), dK and dV by blocks of 64 keys over the
// rows of the group.  Both form S and dP again.  Where there are fewer blocks
// than SMs, the long axis is split and the partial sums are added afterwards.
// Rows and keys past the end are loaded as zeros, so that nothing there can
// reach a product.
#pragma once

#include "../lard_exp2.cuh"
#include "attn_common.cuh"

namespace lard {
namespace attn {

constexpr int kSimtThreads = 128;
constexpr int kSimtTile = 64;  // rows and keys of a tile
constexpr int kSimtPStride = 68;

template <int D>
struct SimtLayout {
    static constexpr int LD = D + 4;  // float4 rows of consecutive keys start 4 banks apart
    static constexpr int TILE = kSimtTile * LD;
    static constexpr int P = kSimtTile * kSimtPStride;
    static constexpr int FWD_BYTES = (5 * TILE + P) * 4;   // Q, K and V twice
    static constexpr int DQ_BYTES = (5 * TILE + P) * 4;    // Q, dO, K twice, V
    static constexpr int DKDV_BYTES = (6 * TILE + P) * 4;  // K, V, Q and dO twice
    static_assert(DKDV_BYTES <= 232448, "too much shared memory");
};

// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void copy16_or_0(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Requests rows [0, valid) of a tile of ROWS rows and zeros behind; row(t) gives row t's address.
template <int D, int ROWS, typename RowFn>
__device__ __forceinline__ void simt_fetch(float* dst, int valid, const float* any, RowFn row) {
    constexpr int V = D / 4;
#pragma unroll 4
    for (int e = threadIdx.x; e < ROWS * V; e += kSimtThreads) {
        const int t = e / V, c = (e % V) * 4;
        const bool in = t < valid;
        copy16_or_0(ptx::smem_u32(dst + t * SimtLayout<D>::LD + c), in ? row(t) + c : any, in);
    }
}

// s[a][b] = <A row RT ty + a, B row tx + 16 b>: packed pairs of products, even
// and odd c summed apart, so that no operand has to be rearranged.
template <int D, int RT>
__device__ __forceinline__ void simt_dot(const float* A, const float* B, int ty, int tx, float (&s)[RT][4]) {
    constexpr int LD = SimtLayout<D>::LD;
    float2 acc[RT][4];
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[a][b] = splat2(0.f);
#pragma unroll 2
    for (int c = 0; c < D; c += 4) {
        float4 y[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) y[b] = *reinterpret_cast<const float4*>(B + (tx + 16 * b) * LD + c);
#pragma unroll
        for (int a = 0; a < RT; ++a) {
            const float4 x = *reinterpret_cast<const float4*>(A + (RT * ty + a) * LD + c);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                acc[a][b] = fma2(make_float2(x.x, x.y), make_float2(y[b].x, y[b].y), acc[a][b]);
                acc[a][b] = fma2(make_float2(x.z, x.w), make_float2(y[b].z, y[b].w), acc[a][b]);
            }
        }
    }
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) s[a][b] = acc[a][b].x + acc[a][b].y;
}

// acc[a][.] += sum over t of W[RT ty + a][t] (TRANS: W[t][RT ty + a]) times row t of M.
// acc holds D / 64 groups of 4 columns (two pairs), group u at 64 u + 4 tx.
template <int D, int RT, bool TRANS>
__device__ __forceinline__ void simt_accumulate(const float* W, const float* M, int ty, int tx, float2 (&acc)[RT][D / 32]) {
    constexpr int LD = SimtLayout<D>::LD;
    auto step = [&](int t, const float (&w)[RT]) {
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
            const float4 m = *reinterpret_cast<const float4*>(M + t * LD + 64 * u + 4 * tx);
#pragma unroll
            for (int a = 0; a < RT; ++a) {
                const float2 w2 = splat2(w[a]);
                acc[a][2 * u] = fma2(w2, make_float2(m.x, m.y), acc[a][2 * u]);
                acc[a][2 * u + 1] = fma2(w2, make_float2(m.z, m.w), acc[a][2 * u + 1]);
            }
        }
    };
    if constexpr (TRANS) {
#pragma unroll 2
        for (int t = 0; t < kSimtTile; ++t) {
            float w[RT];
#pragma unroll
            for (int a = 0; a < RT; a += 4) {
                const float4 x = *reinterpret_cast<const float4*>(W + t * kSimtPStride + RT * ty + a);
                w[a] = x.x;
                w[a + 1] = x.y;
                w[a + 2] = x.z;
                w[a + 3] = x.w;
            }
            step(t, w);
        }
    } else {
#pragma unroll 1
        for (int t = 0; t < kSimtTile; t += 4) {
            float w[4][RT];
#pragma unroll
            for (int a = 0; a < RT; ++a) {
                const float4 x = *reinterpret_cast<const float4*>(W + (RT * ty + a) * kSimtPStride + t);
                w[0][a] = x.x;
                w[1][a] = x.y;
                w[2][a] = x.z;
                w[3][a] = x.w;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) step(t + k, w[k]);
        }
    }
}

__device__ __forceinline__ float4 scaled(float2 a, float2 b, float s) { return make_float4(a.x * s, a.y * s, b.x * s, b.y * s); }

// Grid: row tiles of 8 RT rows (fastest), then splits, then problems.
template <int D, int RT>
__global__ void __launch_bounds__(kSimtThreads) attn_fwd_simt_kernel(const __grid_constant__ FwdArgs<float> g) {
    using L = SimtLayout<D>;
    constexpr int kRows = 8 * RT;
    extern __shared__ float4 smem4[];
    float* qs = reinterpret_cast<float*>(smem4);
    float* ks = qs + L::TILE;      // two
    float* vs = ks + 2 * L::TILE;  // two
    float* ps = vs + 2 * L::TILE;
    const int rtiles = (g.R + kRows - 1) / kRows;
    const int r0 = static_cast<int>(blockIdx.x % rtiles) * kRows;
    const int split = static_cast<int>(blockIdx.x / rtiles % g.splits);
    const int ph = static_cast<int>(blockIdx.x / rtiles / g.splits);
    const int pb = ph / g.Hkv, hk = ph % g.Hkv;
    const int Gn = g.G * g.n;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int rows = min(kRows, g.R - r0);

    const int len0 = g.seg[0].length(pb), len1 = g.nseg > 1 ? g.seg[1].length(pb) : 0;
    const int tiles0 = (len0 + kSimtTile - 1) / kSimtTile;
    const long long all = static_cast<long long>(tiles0) + (len1 + kSimtTile - 1) / kSimtTile;
    const int t0 = static_cast<int>(all * split / g.splits), t1 = static_cast<int>(all * (split + 1) / g.splits);
    auto fetch = [&](int t, bool value) {
        const bool second = t >= tiles0;
        const KeySeg<float>& seg = g.seg[second ? 1 : 0];
        const int j0 = (second ? t - tiles0 : t) * kSimtTile;
        const View<const float>& src = value ? seg.v : seg.k;
        simt_fetch<D, kSimtTile>((value ? vs : ks) + (t & 1) * L::TILE, (second ? len1 : len0) - j0, src.p,
                                 [&](int u) { return src.row(pb, hk, j0 + u); });
    };
    simt_fetch<D, kRows>(qs, rows, g.q.p, [&](int t) {
        const int r = r0 + t, rem = r % Gn;
        return g.q.row(pb + r / Gn, hk * g.G + rem / g.n, rem % g.n);
    });
    if (t0 < t1) fetch(t0, false);
    copy_commit();
    if (t0 < t1) fetch(t0, true);
    copy_commit();

    float m[RT], l[RT];
    float2 o[RT][D / 32];
#pragma unroll
    for (int a = 0; a < RT; ++a) {
        m[a] = -INFINITY;
        l[a] = 0.f;
#pragma unroll
        for (int u = 0; u < D / 32; ++u) o[a][u] = splat2(0.f);
    }
    for (int t = t0; t < t1; ++t) {
        const bool second = t >= tiles0;
        const int len = second ? len1 : len0, j0 = (second ? t - tiles0 : t) * kSimtTile;
        const bool causal = g.seg[second ? 1 : 0].causal;
        copy_wait<1>();
        __syncthreads();  // K of this tile is there; the last tile's products are done
        if (t + 1 < t1) fetch(t + 1, false);
        copy_commit();
        float z[RT][4];
        simt_dot<D, RT>(qs, ks + (t & 1) * L::TILE, ty, tx, z);
#pragma unroll
        for (int a = 0; a < RT; ++a) {
            const int lim = causal ? causal_limit(len, g.n, (r0 + RT * ty + a) % g.n) : len;
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (j0 + tx + 16 * c >= lim) z[a][c] = -INFINITY;
                top = fmaxf(top, z[a][c]);
            }
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float mn = fmaxf(m[a], top * g.cfac);
            const float base = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: every exponential below is 0
            const float sc = exp2f(m[a] - base);
            m[a] = mn;
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float p = exp2f(fmaf(z[a][c], g.cfac, -base));
                sum += p;
                ps[(RT * ty + a) * kSimtPStride + tx + 16 * c] = p;
            }
            l[a] = l[a] * sc + sum;  // of this thread's columns
#pragma unroll
            for (int u = 0; u < D / 32; ++u) o[a][u] = mul2(o[a][u], splat2(sc));
        }
        copy_wait<1>();
        __syncthreads();  // V is there, P is written
        if (t + 1 < t1) fetch(t + 1, true);
        copy_commit();
        simt_accumulate<D, RT, false>(ps, vs + (t & 1) * L::TILE, ty, tx, o);
    }
    copy_wait<0>();
#pragma unroll
    for (int a = 0; a < RT; ++a) {
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) l[a] += __shfl_xor_sync(0xffffffffu, l[a], x);
        const int r = r0 + RT * ty + a;
        if (r >= g.R) continue;
        const int b = pb + r / Gn, rem = r % Gn;
        const long long row = (static_cast<long long>(b) * g.Hkv + hk) * Gn + rem;
        const float inv = l[a] == 0.f ? 0.f : 1.f / l[a];
        const float lse = l[a] == 0.f ? -INFINITY : (m[a] + log2f(l[a])) * kLn2;
        float* dst = g.join ? g.part_o + ((g.split0 + split) * g.rows + row) * D : g.out.row(b, hk * g.G + rem / g.n, rem % g.n);
#pragma unroll
        for (int u = 0; u < D / 64; ++u) store4(dst + 64 * u + 4 * tx, scaled(o[a][2 * u], o[a][2 * u + 1], inv));
        if (tx == 0) {
            if (g.join) g.part_lse[(g.split0 + split) * g.rows + row] = lse;
            else g.lse[row] = lse;
        }
    }
}

// Backward work of cross attention; rows and heads as in FwdArgs.
struct SimtBwdArgs {
    View<const float> q, k, v, out, dout;
    View<float> dq, dk, dv;
    const float* lse;  // [B, Hq, n]
    float* delta;      // [B, Hq, n], workspace
    const int* len;
    int m, B, Hkv, G, n;
    // More than one split: sums go to [split][row][D] buffers, rows of dq in the
    // order (b, head, i), of dk and dv in the order (b, key head, j).
    int qsplits, ksplits;
    float *part_q, *part_k, *part_v;
    float cfac, tau;
    __device__ __forceinline__ int length(int b) const {
        if (!len) return m;
        const int l = len[b];
        return l < 0 ? 0 : (l > m ? m : l);
    }
};

// dQ of 64 rows, and their delta = rowsum(dO O).  Grid: row tiles (fastest), splits, B * Hkv.
template <int D>
__global__ void __launch_bounds__(kSimtThreads) attn_dq_simt_kernel(const __grid_constant__ SimtBwdArgs g) {
    using L = SimtLayout<D>;
    constexpr int RT = 8;
    extern __shared__ float4 smem4[];
    float* qs = reinterpret_cast<float*>(smem4);
    float* os = qs + L::TILE;
    float* ks = os + L::TILE;  // two
    float* vs = ks + 2 * L::TILE;
    float* ds = vs + L::TILE;
    const int R = g.G * g.n;
    const int rtiles = (R + kSimtTile - 1) / kSimtTile;
    const int r0 = static_cast<int>(blockIdx.x % rtiles) * kSimtTile;
    const int split = static_cast<int>(blockIdx.x / rtiles % g.qsplits);
    const int bh = static_cast<int>(blockIdx.x / rtiles / g.qsplits);
    const int b = bh / g.Hkv, hk = bh % g.Hkv;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int rows = min(kSimtTile, R - r0), len = g.length(b);
    const int tiles = (len + kSimtTile - 1) / kSimtTile;
    const int t0 = static_cast<int>(static_cast<long long>(tiles) * split / g.qsplits);
    const int t1 = static_cast<int>(static_cast<long long>(tiles) * (split + 1) / g.qsplits);
    auto keys = [&](int t) {
        simt_fetch<D, kSimtTile>(ks + (t & 1) * L::TILE, len - t * kSimtTile, g.k.p,
                                 [&](int u) { return g.k.row(b, hk, t * kSimtTile + u); });
    };
    auto values = [&](int t) {
        simt_fetch<D, kSimtTile>(vs, len - t * kSimtTile, g.v.p, [&](int u) { return g.v.row(b, hk, t * kSimtTile + u); });
    };
    auto head = [&](int t) { return hk * g.G + (r0 + t) / g.n; };
    auto pos = [&](int t) { return (r0 + t) % g.n; };
    simt_fetch<D, kSimtTile>(qs, rows, g.q.p, [&](int t) { return g.q.row(b, head(t), pos(t)); });
    simt_fetch<D, kSimtTile>(os, rows, g.dout.p, [&](int t) { return g.dout.row(b, head(t), pos(t)); });
    if (t0 < t1) keys(t0);
    copy_commit();
    if (t0 < t1) values(t0);
    copy_commit();
    // delta of this thread's rows: 16 lanes share a row.
    float nl2[RT], delta[RT];
#pragma unroll
    for (int a = 0; a < RT; ++a) {
        const int t = RT * ty + a;
        float s = 0.f;
        nl2[a] = 0.f;
        if (t < rows) {
            const float *x = g.dout.row(b, head(t), pos(t)), *y = g.out.row(b, head(t), pos(t));
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                const float4 p = load4(x + 64 * u + 4 * tx), q = load4(y + 64 * u + 4 * tx);
                s = fmaf(p.x, q.x, fmaf(p.y, q.y, fmaf(p.z, q.z, fmaf(p.w, q.w, s))));
            }
            nl2[a] = -g.lse[static_cast<size_t>(bh) * R + r0 + t] * kLog2e;
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        delta[a] = s;
        if (t < rows && tx == 0 && split == 0) g.delta[static_cast<size_t>(bh) * R + r0 + t] = s;
    }
    float2 dq[RT][D / 32];
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int u = 0; u < D / 32; ++u) dq[a][u] = splat2(0.f);
    for (int t = t0; t < t1; ++t) {
        const int j0 = t * kSimtTile;
        const float* kt = ks + (t & 1) * L::TILE;
        copy_wait<1>();
        __syncthreads();  // K is there; the last tile's products are done
        if (t + 1 < t1) keys(t + 1);
        copy_commit();
        float z[RT][4], dp[RT][4];
        simt_dot<D, RT>(qs, kt, ty, tx, z);
        copy_wait<1>();
        __syncthreads();  // V is there
        simt_dot<D, RT>(os, vs, ty, tx, dp);
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const bool seen = RT * ty + a < rows && j0 + tx + 16 * c < len;
                const float p = exp2f(fmaf(z[a][c], g.cfac, nl2[a]));
                ds[(RT * ty + a) * kSimtPStride + tx + 16 * c] = seen ? p * (dp[a][c] - delta[a]) : 0.f;
            }
        __syncthreads();  // dZ is written, V has been read
        if (t + 1 < t1) values(t + 1);
        copy_commit();
        simt_accumulate<D, RT, false>(ds, kt, ty, tx, dq);
    }
    copy_wait<0>();
    const float scale = g.qsplits > 1 ? 1.f : g.tau;
#pragma unroll
    for (int a = 0; a < RT; ++a) {
        const int t = RT * ty + a;
        if (t >= rows) continue;
        float* dst = g.qsplits > 1 ? g.part_q + ((static_cast<size_t>(split) * g.B * g.Hkv + bh) * R + r0 + t) * D
                                   : g.dq.row(b, head(t), pos(t));
#pragma unroll
        for (int u = 0; u < D / 64; ++u) store4(dst + 64 * u + 4 * tx, scaled(dq[a][2 * u], dq[a][2 * u + 1], scale));
    }
}

// dK, dV of 64 keys.  Grid: key tiles of m (fastest), splits, B * Hkv.
template <int D>
__global__ void __launch_bounds__(kSimtThreads) attn_dkdv_simt_kernel(const __grid_constant__ SimtBwdArgs g) {
    using L = SimtLayout<D>;
    constexpr int RT = 8;
    extern __shared__ float4 smem4[];
    float* ks = reinterpret_cast<float*>(smem4);
    float* vs = ks + L::TILE;
    float* qs = vs + L::TILE;      // two
    float* os = qs + 2 * L::TILE;  // two
    float* ps = os + 2 * L::TILE;  // P, then dZ: [row][key]
    const int ktiles = (g.m + kSimtTile - 1) / kSimtTile;
    const int j0 = static_cast<int>(blockIdx.x % ktiles) * kSimtTile;
    const int split = static_cast<int>(blockIdx.x / ktiles % g.ksplits);
    const int bh = static_cast<int>(blockIdx.x / ktiles / g.ksplits);
    const int b = bh / g.Hkv, hk = bh % g.Hkv;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int R = g.G * g.n, len = g.length(b);
    const int tiles = j0 < len ? (R + kSimtTile - 1) / kSimtTile : 0;
    const int t0 = static_cast<int>(static_cast<long long>(tiles) * split / g.ksplits);
    const int t1 = static_cast<int>(static_cast<long long>(tiles) * (split + 1) / g.ksplits);
    auto fetch = [&](int t, const View<const float>& src, float* dst) {
        const int r0 = t * kSimtTile;
        simt_fetch<D, kSimtTile>(dst + (t & 1) * L::TILE, R - r0, src.p,
                                 [&](int u) { return src.row(b, hk * g.G + (r0 + u) / g.n, (r0 + u) % g.n); });
    };
    if (t0 < t1) {
        simt_fetch<D, kSimtTile>(ks, len - j0, g.k.p, [&](int t) { return g.k.row(b, hk, j0 + t); });
        simt_fetch<D, kSimtTile>(vs, len - j0, g.v.p, [&](int t) { return g.v.row(b, hk, j0 + t); });
        fetch(t0, g.q, qs);
    }
    copy_commit();
    if (t0 < t1) fetch(t0, g.dout, os);
    copy_commit();
    float2 dk[RT][D / 32], dv[RT][D / 32];
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int u = 0; u < D / 32; ++u) dk[a][u] = dv[a][u] = splat2(0.f);
    for (int t = t0; t < t1; ++t) {
        const int r0 = t * kSimtTile;
        const float *qt = qs + (t & 1) * L::TILE, *ot = os + (t & 1) * L::TILE;
        copy_wait<1>();
        __syncthreads();  // Q is there; the last tile's products are done
        if (t + 1 < t1) fetch(t + 1, g.q, qs);
        copy_commit();
        float z[RT][4], dp[RT][4];
        simt_dot<D, RT>(qt, ks, ty, tx, z);
        copy_wait<1>();
        __syncthreads();  // dO is there
        if (t + 1 < t1) fetch(t + 1, g.dout, os);
        copy_commit();
        simt_dot<D, RT>(ot, vs, ty, tx, dp);
#pragma unroll
        for (int a = 0; a < RT; ++a) {
            const int r = r0 + RT * ty + a;
            const size_t at = static_cast<size_t>(bh) * R + (r < R ? r : 0);
            const float nl2 = -g.lse[at] * kLog2e, delta = g.delta[at];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const bool seen = r < R && j0 + tx + 16 * c < len;
                const float p = seen ? exp2f(fmaf(z[a][c], g.cfac, nl2)) : 0.f;
                ps[(RT * ty + a) * kSimtPStride + tx + 16 * c] = p;
                z[a][c] = p * (dp[a][c] - delta);
            }
        }
        __syncthreads();
        simt_accumulate<D, RT, true>(ps, ot, ty, tx, dv);
        __syncthreads();  // P has been read
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
            for (int c = 0; c < 4; ++c) ps[(RT * ty + a) * kSimtPStride + tx + 16 * c] = z[a][c];
        __syncthreads();
        simt_accumulate<D, RT, true>(ps, qt, ty, tx, dk);
    }
    copy_wait<0>();
    const bool part = g.ksplits > 1;
#pragma unroll
    for (int a = 0; a < RT; ++a) {
        const int j = j0 + RT * ty + a;
        if (j >= g.m) continue;
        const size_t prow = ((static_cast<size_t>(split) * g.B * g.Hkv + bh) * g.m + j) * D;
        float* pk = part ? g.part_k + prow : g.dk.row(b, hk, j);
        float* pv = part ? g.part_v + prow : g.dv.row(b, hk, j);
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
            store4(pk + 64 * u + 4 * tx, scaled(dk[a][2 * u], dk[a][2 * u + 1], part ? 1.f : g.tau));
            store4(pv + 64 * u + 4 * tx, scaled(dv[a][2 * u], dv[a][2 * u + 1], 1.f));
        }
    }
}

}  // namespace attn
}  // namespace lard
