// attn_simt.cuh -- attention of fp32 tensors, on the CUDA cores.
//
// The tensor cores would round fp32 operands, so the products run on the FMA
// pipe, which bounds them (128 multiply-adds a cycle and SM).  A thread owns 4 x
// 4 logits of a 64 x 64 tile (1 x 4 of a 16 x 64 tile where there are few rows)
// and packs multiply-adds in pairs.  256 threads do a tile; a block has two such
// groups at different work, so that each scheduler has four warps, and tiles
// arrive by cp.async meanwhile.  (8 x 4 logits a thread halve the shared-memory
// traffic and the warps: 10 % slower.  The same 4 x 4 with a warp's threads 4 x 8
// in place of 2 x 16, two thirds of the traffic: 2 % slower.)
// Measured, 8 heads of 1000 x 2000 rows at d = 128: forward 278 us (29.5 TFLOP/s, the
// FMA pipe busy 51 % of the time, 59 % on the 128 of 148 SMs that have a block), dQ 391 us
// (52 %), dK and dV 491 us (56 %), their sums 20 us.
// Forward: the groups take alternate key tiles and are joined at the end; running row
// maximum and sum in the log2 domain, P through shared memory, O in registers.
// Backward: one kernel for each side of the logits, so that every sum has one
// owner and a fixed order (no atomics): dQ by blocks of 64 rows over the keys (it
// also forms delta), dK and dV by blocks of 64 keys over the rows of the group.
// Group 0 forms S and P, group 1 dP and dZ; then each takes half of dQ's keys, or
// group 0 dV and group 1 dK.  Where there are fewer blocks than SMs, the long
// axis is split and the partial sums are added afterwards.
// Rows and keys past the end are loaded as zeros, so that nothing there can
// reach a product.
#pragma once

#include "../lard_exp2.cuh"
#include "attn_common.cuh"
#include "attn_ptx.cuh"

namespace lard {
namespace attn {

constexpr int kSimtGroup = 256, kSimtThreads = 2 * kSimtGroup;
constexpr int kSimtTile = 64;  // rows and keys of a tile
constexpr int kSimtPStride = 68;

template <int D>
struct SimtLayout {
    static constexpr int LD = D + 4;  // float4 rows of consecutive keys start 4 banks apart
    static constexpr int TILE = kSimtTile * LD;
    static constexpr int P = kSimtTile * kSimtPStride;
    static constexpr int FWD_BYTES = (5 * TILE + 2 * P) * 4;   // Q; K, V and P of each group
    static constexpr int DQ_BYTES = (5 * TILE + P) * 4;        // Q, dO, K twice, V; P, then dZ
    static constexpr int DKDV_BYTES = (4 * TILE + 2 * P) * 4;  // K, V, Q, dO; P, dZ
    static_assert(FWD_BYTES <= 232448, "too much shared memory");
};

// Requests rows [0, valid) of a tile of ROWS rows and zeros behind; row(t) gives row t's address.
// THREADS threads take part, `me` the number of each.
template <int D, int ROWS, int THREADS, typename RowFn>
__device__ __forceinline__ void simt_fetch(int me, float* dst, int valid, const float* any, RowFn row) {
    constexpr int V = D / 4;
#pragma unroll 4
    for (int e = me; e < ROWS * V; e += THREADS) {
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

// acc[a][.] += sum over t in [T0, T1) of W[RT ty + a][t] (TRANS: W[t][RT ty + a]) times row t of M.
// acc holds D / 64 groups of 4 columns (two pairs), group u at 64 u + 4 tx.
template <int D, int RT, bool TRANS>
__device__ __forceinline__ void simt_accumulate(const float* W, const float* M, int ty, int tx, float2 (&acc)[RT][D / 32],
                                                int T0 = 0, int T1 = kSimtTile) {
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
        for (int t = T0; t < T1; ++t) {
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
        for (int t = T0; t < T1; t += 4) {
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

// Grid: row tiles of 16 RT rows (fastest), then splits, then problems.
template <int D, int RT>
__global__ void __launch_bounds__(kSimtThreads) attn_fwd_simt_kernel(const __grid_constant__ FwdArgs<float> g) {
    using L = SimtLayout<D>;
    if (g.join) next_may_start();
    constexpr int kRows = kSimtGroup / 16 * RT;
    extern __shared__ float4 smem4[];
    const int grp = threadIdx.x / kSimtGroup, me = threadIdx.x % kSimtGroup;
    float* qs = reinterpret_cast<float*>(smem4);
    float* ks = qs + L::TILE + grp * (2 * L::TILE + L::P);
    float* vs = ks + L::TILE;
    float* ps = vs + L::TILE;
    const int rtiles = (g.R + kRows - 1) / kRows;
    const int r0 = static_cast<int>(blockIdx.x % rtiles) * kRows;
    const int split = static_cast<int>(blockIdx.x / rtiles % g.splits);
    const int ph = static_cast<int>(blockIdx.x / rtiles / g.splits);
    const int pb = ph / g.Hkv, hk = ph % g.Hkv;
    const int Gn = g.G * g.n;
    const int tx = me & 15, ty = me >> 4;
    const int rows = min(kRows, g.R - r0);

    const int len0 = g.seg[0].length(pb), len1 = g.nseg > 1 ? g.seg[1].length(pb) : 0;
    const int tiles0 = (len0 + kSimtTile - 1) / kSimtTile;
    const long long all = static_cast<long long>(tiles0) + (len1 + kSimtTile - 1) / kSimtTile;
    const int t0 = static_cast<int>(all * split / g.splits) + grp, t1 = static_cast<int>(all * (split + 1) / g.splits);
    auto fetch = [&](int t, bool value) {
        const bool second = t >= tiles0;
        const KeySeg<float>& seg = g.seg[second ? 1 : 0];
        const int j0 = (second ? t - tiles0 : t) * kSimtTile;
        const View<const float>& src = value ? seg.v : seg.k;
        simt_fetch<D, kSimtTile, kSimtGroup>(me, value ? vs : ks, (second ? len1 : len0) - j0, src.p,
                                             [&](int u) { return src.row(pb, hk, j0 + u); });
    };
    simt_fetch<D, kRows, kSimtThreads>(threadIdx.x, qs, rows, g.q.p, [&](int t) {
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
    copy_wait<1>();
    __syncthreads();  // Q is there, brought by both groups
    for (int t = t0; t < t1; t += 2) {
        const bool second = t >= tiles0;
        const int len = second ? len1 : len0, j0 = (second ? t - tiles0 : t) * kSimtTile;
        const bool causal = g.seg[second ? 1 : 0].causal;
        copy_wait<1>();
        ptx::named_bar_sync(1 + grp, kSimtGroup);  // K of this tile is there; the last tile's products are done
        float z[RT][4];
        simt_dot<D, RT>(qs, ks, ty, tx, z);
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
        copy_wait<0>();
        ptx::named_bar_sync(1 + grp, kSimtGroup);  // V is there, P is written, K has been read
        if (t + 2 < t1) fetch(t + 2, false);
        copy_commit();
        simt_accumulate<D, RT, false>(ps, vs, ty, tx, o);
        ptx::named_bar_sync(1 + grp, kSimtGroup);  // V has been read
        if (t + 2 < t1) fetch(t + 2, true);
        copy_commit();
    }
    copy_wait<0>();
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) l[a] += __shfl_xor_sync(0xffffffffu, l[a], x);
    // Group 1 leaves its rows where its tiles were, group 0 joins them to its own.
    float* jo = qs + 3 * L::TILE + L::P;
    float* jm = jo + L::TILE;
    __syncthreads();
    if (grp == 1) {
#pragma unroll
        for (int a = 0; a < RT; ++a) {
            const int t = RT * ty + a;
#pragma unroll
            for (int u = 0; u < D / 64; ++u) store4(jo + t * L::LD + 64 * u + 4 * tx, scaled(o[a][2 * u], o[a][2 * u + 1], 1.f));
            if (tx == 0) {
                jm[2 * t] = m[a];
                jm[2 * t + 1] = l[a];
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int a = 0; a < RT; ++a) {
        const int t = RT * ty + a, r = r0 + t;
        if (grp == 1 || r >= g.R) continue;
        const float m1 = jm[2 * t], top = fmaxf(m[a], m1), base = top == -INFINITY ? 0.f : top;
        float w0 = exp2f(m[a] - base), w1 = exp2f(m1 - base);
        const float sum = l[a] * w0 + jm[2 * t + 1] * w1;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const float lse = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
        w0 *= inv;
        w1 *= inv;
        const int b = pb + r / Gn, rem = r % Gn;
        const long long row = (static_cast<long long>(b) * g.Hkv + hk) * Gn + rem;
        float* dst = g.join ? g.part_o + ((g.split0 + split) * g.rows + row) * D : g.out.row(b, hk * g.G + rem / g.n, rem % g.n);
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
            const float4 x = scaled(o[a][2 * u], o[a][2 * u + 1], w0), y = load4(jo + t * L::LD + 64 * u + 4 * tx);
            store4(dst + 64 * u + 4 * tx, make_float4(fmaf(y.x, w1, x.x), fmaf(y.y, w1, x.y), fmaf(y.z, w1, x.z), fmaf(y.w, w1, x.w)));
        }
        if (tx == 0) {
            if (g.join) g.part_lse[(g.split0 + split) * g.rows + row] = lse;
            else g.lse[row] = lse;
        }
    }
    if (g.second) wait_for_kernel_before();  // whoever waits for this pass has waited for the first
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
    next_may_start();
    constexpr int RT = 4;
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
    const int grp = threadIdx.x / kSimtGroup, me = threadIdx.x % kSimtGroup;
    const int tx = me & 15, ty = me >> 4;
    const int rows = min(kSimtTile, R - r0), len = g.length(b);
    const int tiles = (len + kSimtTile - 1) / kSimtTile;
    const int t0 = static_cast<int>(static_cast<long long>(tiles) * split / g.qsplits);
    const int t1 = static_cast<int>(static_cast<long long>(tiles) * (split + 1) / g.qsplits);
    auto keys = [&](int t) {
        simt_fetch<D, kSimtTile, kSimtThreads>(threadIdx.x, ks + (t & 1) * L::TILE, len - t * kSimtTile, g.k.p,
                                 [&](int u) { return g.k.row(b, hk, t * kSimtTile + u); });
    };
    auto values = [&](int t) {
        simt_fetch<D, kSimtTile, kSimtThreads>(threadIdx.x, vs, len - t * kSimtTile, g.v.p, [&](int u) { return g.v.row(b, hk, t * kSimtTile + u); });
    };
    auto head = [&](int t) { return hk * g.G + (r0 + t) / g.n; };
    auto pos = [&](int t) { return (r0 + t) % g.n; };
    simt_fetch<D, kSimtTile, kSimtThreads>(threadIdx.x, qs, rows, g.q.p, [&](int t) { return g.q.row(b, head(t), pos(t)); });
    simt_fetch<D, kSimtTile, kSimtThreads>(threadIdx.x, os, rows, g.dout.p, [&](int t) { return g.dout.row(b, head(t), pos(t)); });
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
        if (t < rows && tx == 0 && split == 0 && grp == 0) g.delta[static_cast<size_t>(bh) * R + r0 + t] = s;
    }
    float2 dq[RT][D / 32];
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int u = 0; u < D / 32; ++u) dq[a][u] = splat2(0.f);
    for (int t = t0; t < t1; ++t) {
        const int j0 = t * kSimtTile;
        const float* kt = ks + (t & 1) * L::TILE;
        copy_wait<0>();
        __syncthreads();  // K and V are there; the last tile's products are done
        if (t + 1 < t1) keys(t + 1);
        copy_commit();
        // The two groups' threads of one place (ty, tx) hold the same logits' S and dP.
        float z[RT][4];
        simt_dot<D, RT>(grp ? os : qs, grp ? vs : kt, ty, tx, z);
        if (grp == 0) {
#pragma unroll
            for (int a = 0; a < RT; ++a)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const bool seen = RT * ty + a < rows && j0 + tx + 16 * c < len;
                    const float p = exp2f(fmaf(z[a][c], g.cfac, nl2[a]));
                    ds[(RT * ty + a) * kSimtPStride + tx + 16 * c] = seen ? p : 0.f;
                }
        }
        __syncthreads();  // P is written, V has been read
        if (t + 1 < t1) values(t + 1);
        copy_commit();
        if (grp == 1) {
#pragma unroll
            for (int a = 0; a < RT; ++a)
#pragma unroll
                for (int c = 0; c < 4; ++c) ds[(RT * ty + a) * kSimtPStride + tx + 16 * c] *= z[a][c] - delta[a];
        }
        __syncthreads();  // dZ is written
        simt_accumulate<D, RT, false>(ds, kt, ty, tx, dq, grp * (kSimtTile / 2), (grp + 1) * (kSimtTile / 2));
    }
    copy_wait<0>();
    // Group 0 adds group 1's half of the keys to its own.
    __syncthreads();
    if (grp == 1) {
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
            for (int u = 0; u < D / 64; ++u)
                store4(qs + (RT * ty + a) * L::LD + 64 * u + 4 * tx, scaled(dq[a][2 * u], dq[a][2 * u + 1], 1.f));
    }
    __syncthreads();
    if (grp == 1) return;
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
            const float4 x = load4(qs + (RT * ty + a) * L::LD + 64 * u + 4 * tx);
            dq[a][2 * u] = add2(dq[a][2 * u], make_float2(x.x, x.y));
            dq[a][2 * u + 1] = add2(dq[a][2 * u + 1], make_float2(x.z, x.w));
        }
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
    if (g.qsplits > 1 || g.ksplits > 1) next_may_start();
    constexpr int RT = 4;
    extern __shared__ float4 smem4[];
    float* ks = reinterpret_cast<float*>(smem4);
    float* vs = ks + L::TILE;
    float* qs = vs + L::TILE;
    float* os = qs + L::TILE;
    float* ps = os + L::TILE;  // P: [row][key]
    float* ds = ps + L::P;     // dZ
    const int ktiles = (g.m + kSimtTile - 1) / kSimtTile;
    const int j0 = static_cast<int>(blockIdx.x % ktiles) * kSimtTile;
    const int split = static_cast<int>(blockIdx.x / ktiles % g.ksplits);
    const int bh = static_cast<int>(blockIdx.x / ktiles / g.ksplits);
    const int b = bh / g.Hkv, hk = bh % g.Hkv;
    const int grp = threadIdx.x / kSimtGroup, me = threadIdx.x % kSimtGroup;
    const int tx = me & 15, ty = me >> 4;
    const int R = g.G * g.n, len = g.length(b);
    const int tiles = j0 < len ? (R + kSimtTile - 1) / kSimtTile : 0;
    const int t0 = static_cast<int>(static_cast<long long>(tiles) * split / g.ksplits);
    const int t1 = static_cast<int>(static_cast<long long>(tiles) * (split + 1) / g.ksplits);
    auto fetch = [&](int t, const View<const float>& src, float* dst) {
        const int r0 = t * kSimtTile;
        simt_fetch<D, kSimtTile, kSimtThreads>(threadIdx.x, dst, R - r0, src.p, [&](int u) {
            return src.row(b, hk * g.G + (r0 + u) / g.n, (r0 + u) % g.n);
        });
    };
    if (t0 < t1) {
        simt_fetch<D, kSimtTile, kSimtThreads>(threadIdx.x, ks, len - j0, g.k.p, [&](int t) { return g.k.row(b, hk, j0 + t); });
        simt_fetch<D, kSimtTile, kSimtThreads>(threadIdx.x, vs, len - j0, g.v.p, [&](int t) { return g.v.row(b, hk, j0 + t); });
    }
    wait_for_kernel_before();  // delta
    float2 acc[RT][D / 32];  // group 0: dV, group 1: dK
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
        for (int u = 0; u < D / 32; ++u) acc[a][u] = splat2(0.f);
    for (int t = t0; t < t1; ++t) {
        const int r0 = t * kSimtTile;
        __syncthreads();  // the last tile's products are done
        fetch(t, g.q, qs);
        fetch(t, g.dout, os);
        copy_commit();
        float stat[RT];  // group 0: -LSE log2(e), group 1: delta
#pragma unroll
        for (int a = 0; a < RT; ++a) {
            const int r = r0 + RT * ty + a;
            const size_t at = static_cast<size_t>(bh) * R + (r < R ? r : 0);
            stat[a] = grp ? g.delta[at] : -g.lse[at] * kLog2e;
        }
        copy_wait<0>();
        __syncthreads();
        float z[RT][4];
        simt_dot<D, RT>(grp ? os : qs, grp ? vs : ks, ty, tx, z);
        if (grp == 0) {
#pragma unroll
            for (int a = 0; a < RT; ++a)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const bool seen = r0 + RT * ty + a < R && j0 + tx + 16 * c < len;
                    ps[(RT * ty + a) * kSimtPStride + tx + 16 * c] = seen ? exp2f(fmaf(z[a][c], g.cfac, stat[a])) : 0.f;
                }
        }
        __syncthreads();  // P is written
        if (grp == 1) {
#pragma unroll
            for (int a = 0; a < RT; ++a)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int at = (RT * ty + a) * kSimtPStride + tx + 16 * c;
                    ds[at] = ps[at] * (z[a][c] - stat[a]);
                }
            ptx::named_bar_sync(1, kSimtGroup);
        }
        simt_accumulate<D, RT, true>(grp ? ds : ps, grp ? qs : os, ty, tx, acc);
    }
    copy_wait<0>();
    const bool part = g.ksplits > 1;
#pragma unroll
    for (int a = 0; a < RT; ++a) {
        const int j = j0 + RT * ty + a;
        if (j >= g.m) continue;
        const size_t prow = ((static_cast<size_t>(split) * g.B * g.Hkv + bh) * g.m + j) * D;
        float* dst = part ? (grp ? g.part_k : g.part_v) + prow : (grp ? g.dk : g.dv).row(b, hk, j);
#pragma unroll
        for (int u = 0; u < D / 64; ++u)  // zeros past the length, whatever dO holds
            store4(dst + 64 * u + 4 * tx, j < len ? scaled(acc[a][2 * u], acc[a][2 * u + 1], grp && !part ? g.tau : 1.f)
                                                  : make_float4(0.f, 0.f, 0.f, 0.f));
    }
}

}  // namespace attn
}  // namespace lard
