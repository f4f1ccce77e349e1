// attn_simt.cuh -- attention on the CUDA cores, in fp32.
//
// Forward: a block owns 64 query rows of one (sequence, key head) and streams
// 64-key tiles: S = Q K^T in registers (4 x 4 per thread), running row maximum
// and sum in the log2 domain, P through shared memory, O += P V in registers.
// Backward: one kernel per gradient side, so that every sum has one owner and
// a fixed order (no atomics): dK, dV by blocks of 64 keys over all rows of the
// group, dQ by blocks of 64 rows over all keys.  Both form S and dP again.
// Rows and keys past the end are loaded as zeros, so that nothing there can
// reach a product.
#pragma once

#include "attn_common.cuh"

namespace lard {
namespace attn {

constexpr int kSimtThreads = 256;
constexpr int kSimtTile = 64;   // rows and keys of a tile
constexpr int kSimtPStride = 68;

template <int D>
struct SimtLayout {
    static constexpr int LD = D + 4;  // float4 rows of consecutive keys start 4 banks apart
    static constexpr int TILE = kSimtTile * LD;
    static constexpr int P = kSimtTile * kSimtPStride;
    static constexpr int FWD_BYTES = (2 * TILE + P) * 4;
    static constexpr int BWD_BYTES = (4 * TILE + 2 * P) * 4;
};

// Loads rows [0, valid) of a 64-row tile and zeros behind; row(t) gives row t's address.
template <int D, typename T, typename RowFn>
__device__ __forceinline__ void simt_load_tile(float* dst, int valid, RowFn row) {
    constexpr int V = D / 4;
    for (int e = threadIdx.x; e < kSimtTile * V; e += kSimtThreads) {
        const int t = e / V, c = (e % V) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < valid) x = load4(row(t) + c);
        *reinterpret_cast<float4*>(dst + t * SimtLayout<D>::LD + c) = x;
    }
}

// s[a][b] = <A row 4 ty + a, B row tx + 16 b>.
template <int D>
__device__ __forceinline__ void simt_dot(const float* A, const float* B, int ty, int tx, float (&s)[4][4]) {
    constexpr int LD = SimtLayout<D>::LD;
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) s[a][b] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) x[a] = *reinterpret_cast<const float4*>(A + (4 * ty + a) * LD + c);
#pragma unroll
        for (int b = 0; b < 4; ++b) y[b] = *reinterpret_cast<const float4*>(B + (tx + 16 * b) * LD + c);
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                s[a][b] = fmaf(x[a].x, y[b].x, s[a][b]);
                s[a][b] = fmaf(x[a].y, y[b].y, s[a][b]);
                s[a][b] = fmaf(x[a].z, y[b].z, s[a][b]);
                s[a][b] = fmaf(x[a].w, y[b].w, s[a][b]);
            }
    }
}

// acc[a][.] += sum over t of W[t][4 ty + a] (columns: TRANS) or W[4 ty + a][t] times row t of M.
// acc holds D / 64 groups of 4 columns, group u at 64 u + 4 tx.
template <int D, bool TRANS>
__device__ __forceinline__ void simt_accumulate(const float* W, const float* M, int ty, int tx,
                                                float (&acc)[4][D / 16]) {
    constexpr int LD = SimtLayout<D>::LD;
#pragma unroll 2
    for (int t = 0; t < kSimtTile; t += 4) {
        float w[4][4];  // [a][step]
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 x = *reinterpret_cast<const float4*>(
                TRANS ? W + (t + k) * kSimtPStride + 4 * ty : W + (4 * ty + k) * kSimtPStride + t);
            if (TRANS) { w[0][k] = x.x; w[1][k] = x.y; w[2][k] = x.z; w[3][k] = x.w; }
            else { w[k][0] = x.x; w[k][1] = x.y; w[k][2] = x.z; w[k][3] = x.w; }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                const float4 m = *reinterpret_cast<const float4*>(M + (t + k) * LD + 64 * u + 4 * tx);
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    acc[a][4 * u] = fmaf(w[a][k], m.x, acc[a][4 * u]);
                    acc[a][4 * u + 1] = fmaf(w[a][k], m.y, acc[a][4 * u + 1]);
                    acc[a][4 * u + 2] = fmaf(w[a][k], m.z, acc[a][4 * u + 2]);
                    acc[a][4 * u + 3] = fmaf(w[a][k], m.w, acc[a][4 * u + 3]);
                }
            }
    }
}

// Grid: row tiles (fastest), then splits, then B * Hkv.
template <typename T, int D>
__global__ void __launch_bounds__(kSimtThreads) attn_fwd_simt_kernel(const __grid_constant__ FwdArgs<T> g) {
    using L = SimtLayout<D>;
    extern __shared__ float4 smem4[];
    float* qs = reinterpret_cast<float*>(smem4);
    float* kv = qs + L::TILE;
    float* ps = kv + L::TILE;
    const int R = g.G * g.n;
    const int rtiles = (R + kSimtTile - 1) / kSimtTile;
    const int r0 = static_cast<int>(blockIdx.x % rtiles) * kSimtTile;
    const int split = static_cast<int>(blockIdx.x / rtiles % g.splits);
    const int bh = static_cast<int>(blockIdx.x / rtiles / g.splits);
    const int b = bh / g.Hkv, hk = bh % g.Hkv;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int rows = min(kSimtTile, R - r0);

    simt_load_tile<D, T>(qs, rows, [&](int t) {
        const int r = r0 + t;
        return g.q.row(b, hk * g.G + r / g.n, r % g.n);
    });
    int len[2] = {0, 0}, tiles[2] = {0, 0};
    for (int s = 0; s < g.nseg; ++s) {
        len[s] = g.seg[s].length(b);
        tiles[s] = (len[s] + kSimtTile - 1) / kSimtTile;
    }
    const long long T_all = static_cast<long long>(tiles[0]) + tiles[1];
    const long long t0 = T_all * split / g.splits, t1 = T_all * (split + 1) / g.splits;

    float m[4], l[4], o[4][D / 16];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        m[a] = -INFINITY;
        l[a] = 0.f;
#pragma unroll
        for (int u = 0; u < D / 16; ++u) o[a][u] = 0.f;
    }
    for (long long t = t0; t < t1; ++t) {
        const int s = t < tiles[0] ? 0 : 1;
        const KeySeg<T>& seg = g.seg[s];
        const int j0 = static_cast<int>(s == 0 ? t : t - tiles[0]) * kSimtTile;
        const int valid = min(kSimtTile, len[s] - j0);
        __syncthreads();  // the last tile's V has been read
        simt_load_tile<D, T>(kv, valid, [&](int u) { return seg.k.row(b, hk, j0 + u); });
        __syncthreads();
        float z[4][4];
        simt_dot<D>(qs, kv, ty, tx, z);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const int r = r0 + 4 * ty + a;
            const int lim = seg.causal ? causal_limit(len[s], g.n, r % g.n) : len[s];
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
                ps[(4 * ty + a) * kSimtPStride + tx + 16 * c] = p;
            }
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            l[a] = l[a] * sc + sum;
#pragma unroll
            for (int u = 0; u < D / 16; ++u) o[a][u] *= sc;
        }
        __syncthreads();  // K has been read, P is written
        simt_load_tile<D, T>(kv, valid, [&](int u) { return seg.v.row(b, hk, j0 + u); });
        __syncthreads();
        simt_accumulate<D, false>(ps, kv, ty, tx, o);
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const int r = r0 + 4 * ty + a;
        if (r >= R) continue;
        const float inv = l[a] > 0.f ? 1.f / l[a] : (l[a] == 0.f ? 0.f : l[a]);
        const float lse = l[a] == 0.f ? -INFINITY : (m[a] + log2f(l[a])) * kLn2;
        if (g.splits > 1) {
            const size_t pr = (static_cast<size_t>(split) * g.B * g.Hkv + bh) * R + r;
#pragma unroll
            for (int u = 0; u < D / 64; ++u)
                store4(g.part_o + pr * D + 64 * u + 4 * tx,
                       make_float4(o[a][4 * u] * inv, o[a][4 * u + 1] * inv, o[a][4 * u + 2] * inv, o[a][4 * u + 3] * inv));
            if (tx == 0) g.part_lse[pr] = lse;
        } else {
            T* dst = g.out.row(b, hk * g.G + r / g.n, r % g.n);
#pragma unroll
            for (int u = 0; u < D / 64; ++u)
                store4(dst + 64 * u + 4 * tx,
                       make_float4(o[a][4 * u] * inv, o[a][4 * u + 1] * inv, o[a][4 * u + 2] * inv, o[a][4 * u + 3] * inv));
            if (tx == 0) g.lse[static_cast<size_t>(bh) * R + r] = lse;
        }
    }
}

// Joins the splits of a row: LSE = log sum_s exp LSE_s, O = sum_s exp(LSE_s - LSE) O_s.
// One warp per row; lanes share the head dimension.
template <typename T, int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ FwdArgs<T> g) {
    const int lane = threadIdx.x & 31;
    const long long rows = static_cast<long long>(g.B) * g.Hkv * g.G * g.n;
    const long long row = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (row >= rows) return;
    constexpr int E = D / 32;
    float top = -INFINITY;
    for (int s = lane; s < g.splits; s += 32) top = fmaxf(top, g.part_lse[s * rows + row]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float base = top == -INFINITY ? 0.f : top;
    float total = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int s = 0; s < g.splits; ++s) {
        const float w = exp2f((g.part_lse[s * rows + row] - base) * kLog2e);
        total += w;
        if (w == 0.f) continue;  // a split that saw nothing need not have written its O
        const float* src = g.part_o + (s * rows + row) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(w, src[e], o[e]);
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const int R = g.G * g.n;
    const int bh = static_cast<int>(row / R), r = static_cast<int>(row % R);
    T* dst = g.out.row(bh / g.Hkv, bh % g.Hkv * g.G + r / g.n, r % g.n) + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = static_cast<T>(o[e] * inv);
    if (lane == 0) g.lse[row] = total == 0.f ? -INFINITY : base + log2f(total) * kLn2;
}

// Backward work of cross attention; rows and heads as in FwdArgs.
template <typename T>
struct BwdArgs {
    View<const T> q, k, v, out, dout;
    View<T> dq, dk, dv;
    const float* lse;  // [B, Hq, n]
    float* delta;      // [B, Hq, n], workspace
    const int* len;
    int m;
    int B, Hkv, G, n;
    float cfac, tau;
    __device__ __forceinline__ int length(int b) const {
        if (!len) return m;
        const int l = len[b];
        return l < 0 ? 0 : (l > m ? m : l);
    }
};

// delta = rowsum(dO * O), one warp per row.
template <typename T, int D>
__global__ void __launch_bounds__(256) attn_delta_kernel(const __grid_constant__ BwdArgs<T> g) {
    const int lane = threadIdx.x & 31;
    const int R = g.G * g.n;
    const long long row = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (row >= static_cast<long long>(g.B) * g.Hkv * R) return;
    const int bh = static_cast<int>(row / R), r = static_cast<int>(row % R);
    const int b = bh / g.Hkv, h = bh % g.Hkv * g.G + r / g.n, i = r % g.n;
    float s = 0.f;
    if (lane * 4 < D) {
        const float4 x = load4(g.dout.row(b, h, i) + lane * 4), y = load4(g.out.row(b, h, i) + lane * 4);
        s = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, x.w * y.w)));
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    if (lane == 0) g.delta[row] = s;
}

// The probabilities and dZ of a 64 x 64 tile into shared memory ([row][key]), from S and dP.
// Rows past the end have zeros in both tiles of operands and are written as 0; so are masked keys.
template <typename T>
__device__ __forceinline__ void simt_probs(const BwdArgs<T>& g, int bh, int r0, int R, int j0, int len, int ty, int tx,
                                           const float (&z)[4][4], const float (&dp)[4][4], float* ps, float* ds) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const int r = r0 + 4 * ty + a;
        float lse2 = 0.f, delta = 0.f;
        if (r < R) {
            lse2 = g.lse[static_cast<size_t>(bh) * R + r] * kLog2e;
            delta = g.delta[static_cast<size_t>(bh) * R + r];
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const bool seen = r < R && j0 + tx + 16 * c < len;
            const float p = seen ? exp2f(fmaf(z[a][c], g.cfac, -lse2)) : 0.f;
            const int at = (4 * ty + a) * kSimtPStride + tx + 16 * c;
            if (ps) ps[at] = p;
            ds[at] = seen ? p * (dp[a][c] - delta) : 0.f;
        }
    }
}

// dK, dV of 64 keys.  Grid: key tiles of m (fastest), then B * Hkv.
template <typename T, int D>
__global__ void __launch_bounds__(kSimtThreads) attn_dkdv_simt_kernel(const __grid_constant__ BwdArgs<T> g) {
    using L = SimtLayout<D>;
    extern __shared__ float4 smem4[];
    float* ks = reinterpret_cast<float*>(smem4);
    float* vs = ks + L::TILE;
    float* qs = vs + L::TILE;
    float* os = qs + L::TILE;
    float* ps = os + L::TILE;
    float* ds = ps + L::P;
    const int ktiles = (g.m + kSimtTile - 1) / kSimtTile;
    const int j0 = static_cast<int>(blockIdx.x % ktiles) * kSimtTile;
    const int bh = static_cast<int>(blockIdx.x / ktiles);
    const int b = bh / g.Hkv, hk = bh % g.Hkv;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int R = g.G * g.n, len = g.length(b);
    float dk[4][D / 16], dv[4][D / 16];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int u = 0; u < D / 16; ++u) dk[a][u] = dv[a][u] = 0.f;
    if (j0 < len) {
        const int valid = min(kSimtTile, len - j0);
        simt_load_tile<D, T>(ks, valid, [&](int t) { return g.k.row(b, hk, j0 + t); });
        simt_load_tile<D, T>(vs, valid, [&](int t) { return g.v.row(b, hk, j0 + t); });
        for (int r0 = 0; r0 < R; r0 += kSimtTile) {
            const int rows = min(kSimtTile, R - r0);
            __syncthreads();
            simt_load_tile<D, T>(qs, rows, [&](int t) { return g.q.row(b, hk * g.G + (r0 + t) / g.n, (r0 + t) % g.n); });
            simt_load_tile<D, T>(os, rows, [&](int t) { return g.dout.row(b, hk * g.G + (r0 + t) / g.n, (r0 + t) % g.n); });
            __syncthreads();
            float z[4][4], dp[4][4];
            simt_dot<D>(qs, ks, ty, tx, z);
            simt_dot<D>(os, vs, ty, tx, dp);
            simt_probs(g, bh, r0, R, j0, len, ty, tx, z, dp, ps, ds);
            __syncthreads();
            simt_accumulate<D, true>(ps, os, ty, tx, dv);
            simt_accumulate<D, true>(ds, qs, ty, tx, dk);
        }
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const int j = j0 + 4 * ty + a;
        if (j >= g.m) continue;
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
            store4(g.dk.row(b, hk, j) + 64 * u + 4 * tx,
                   make_float4(dk[a][4 * u] * g.tau, dk[a][4 * u + 1] * g.tau, dk[a][4 * u + 2] * g.tau, dk[a][4 * u + 3] * g.tau));
            store4(g.dv.row(b, hk, j) + 64 * u + 4 * tx,
                   make_float4(dv[a][4 * u], dv[a][4 * u + 1], dv[a][4 * u + 2], dv[a][4 * u + 3]));
        }
    }
}

// dQ of 64 rows.  Grid: row tiles (fastest), then B * Hkv.
template <typename T, int D>
__global__ void __launch_bounds__(kSimtThreads) attn_dq_simt_kernel(const __grid_constant__ BwdArgs<T> g) {
    using L = SimtLayout<D>;
    extern __shared__ float4 smem4[];
    float* qs = reinterpret_cast<float*>(smem4);
    float* os = qs + L::TILE;
    float* ks = os + L::TILE;
    float* vs = ks + L::TILE;
    float* ds = vs + L::TILE;
    const int R = g.G * g.n;
    const int rtiles = (R + kSimtTile - 1) / kSimtTile;
    const int r0 = static_cast<int>(blockIdx.x % rtiles) * kSimtTile;
    const int bh = static_cast<int>(blockIdx.x / rtiles);
    const int b = bh / g.Hkv, hk = bh % g.Hkv;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int rows = min(kSimtTile, R - r0), len = g.length(b);
    simt_load_tile<D, T>(qs, rows, [&](int t) { return g.q.row(b, hk * g.G + (r0 + t) / g.n, (r0 + t) % g.n); });
    simt_load_tile<D, T>(os, rows, [&](int t) { return g.dout.row(b, hk * g.G + (r0 + t) / g.n, (r0 + t) % g.n); });
    float dq[4][D / 16];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int u = 0; u < D / 16; ++u) dq[a][u] = 0.f;
    for (int j0 = 0; j0 < len; j0 += kSimtTile) {
        const int valid = min(kSimtTile, len - j0);
        __syncthreads();
        simt_load_tile<D, T>(ks, valid, [&](int t) { return g.k.row(b, hk, j0 + t); });
        simt_load_tile<D, T>(vs, valid, [&](int t) { return g.v.row(b, hk, j0 + t); });
        __syncthreads();
        float z[4][4], dp[4][4];
        simt_dot<D>(qs, ks, ty, tx, z);
        simt_dot<D>(os, vs, ty, tx, dp);
        simt_probs(g, bh, r0, R, j0, len, ty, tx, z, dp, static_cast<float*>(nullptr), ds);
        __syncthreads();
        simt_accumulate<D, false>(ds, ks, ty, tx, dq);
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const int r = r0 + 4 * ty + a;
        if (r >= R) continue;
#pragma unroll
        for (int u = 0; u < D / 64; ++u)
            store4(g.dq.row(b, hk * g.G + r / g.n, r % g.n) + 64 * u + 4 * tx,
                   make_float4(dq[a][4 * u] * g.tau, dq[a][4 * u + 1] * g.tau, dq[a][4 * u + 2] * g.tau, dq[a][4 * u + 3] * g.tau));
    }
}

}  // namespace attn
}  // namespace lard
