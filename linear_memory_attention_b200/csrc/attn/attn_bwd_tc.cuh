// attn_bwd_tc.cuh -- the backward pass on the 5th-generation tensor cores (bf16).
//
// Two kernels, one for each side of the logits, so that every gradient row has
// one owner that sums it in tensor memory in a fixed order: no atomics, no
// fp32 gradient buffers, results that repeat bit for bit.  Both form
// P = 2^(S c - LSE log2 e) and dZ = P (dP - delta) again from the row
// statistics; per 128 x 128 tile that is 3 + 4 products instead of the 5 of a
// kernel that does both sides, but such a kernel has to pass dQ through shared memory
// into fp32 adds in L2, and shared memory bandwidth is what bounds it.
//
// dQ (attn_dq_tc_kernel): a block owns 128 query rows and streams key tiles.
//   S = Q K^T (Q in TMEM), dP = dO V^T, dQ += dZ K (dZ in TMEM, K as MN-major B).
//   It also forms delta = rowsum(dO O) and leaves it for the other kernel.
//   TMEM: Q [0, 64), dZ [64, 128), S [128, 256), dP [256, 384), dQ [384, 384 + D).
//   S and dP are handed back as soon as they are in registers, so the next
//   tile's two products run under this tile's exponentials.
// dK, dV (attn_dkdv_tc_kernel): a block owns 128 keys and streams units of 64
//   query rows of the heads that share them, on transposed tiles (one key a
//   TMEM lane):  S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dZ^T Q, with P^T
//   and dZ^T as TMEM operands in the place of S^T and dP^T.  Two units are in
//   flight, each with a warpgroup of its own.
//   TMEM: dV [0, D), dK [128, 128 + D), S^T of unit u at 256 + 64 (u & 1), dP^T at 384 + 64 (u & 1).
// Per 128 x 128 tile at d = 128 (tensor pipe / shared memory, cycles): dQ 1536 / 1536;
// dK, dV 2048 / 2816, since a 64-row unit reads the resident K and V once each.
// Measured, 4096 rows x 8000 keys, 32 heads, d = 128: dQ 682 us (1.18 PFLOP/s), dK and dV
// 935 us (1.15 PFLOP/s) under the 1000 W cap; the tensor pipe is busy 53 to 55 % of the time in
// either, and what is left is the chain from a product's end to the next one's operands.
// Few blocks (one long axis): the other axis is split so that the SMs are filled once, and
// the partial sums are added in order (attn_join.cuh).
#pragma once

#include "attn_common.cuh"
#include "attn_fwd_tc.cuh"
#include "attn_ptx.cuh"

namespace lard {
namespace attn {

struct TcBwdArgs {
    CUtensorMap k, v;       // boxes of 128 rows
    CUtensorMap q64, do64;  // boxes of 64 rows (dK, dV)
    View<const __nv_bfloat16> q, out, rest, dout;  // rest.p may be NULL
    View<__nv_bfloat16> dq, dk, dv;
    const float* lse;
    float* delta;
    const int* len;
    int m, B, Hkv, G, n;
    // More than one split: sums go to [split][row][D] buffers, rows of dq in the
    // order (b, head, i), of dk and dv in the order (b, key head, j).
    int qsplits, ksplits;
    float *part_q, *part_k, *part_v;
    int khead, kbatch, vhead, vbatch, qhead, qbatch, dohead, dobatch;  // 0 where one block is shared
    float cfac, tau;
    unsigned long long wait_ns, drain_ns;
    __device__ __forceinline__ int length(int b) const {
        if (!len) return m;
        const int l = len[b];
        return l < 0 ? 0 : (l > m ? m : l);
    }
};

constexpr int kBwdTcThreads = 384;

// ---------------------------------------------------------------------- dQ
template <int D>
struct DqLayout {
    static constexpr int KC = D / 64;
    static constexpr int TILE = KC * 16384;
    static constexpr int NK = 3, NV = 2;  // stages of the K and V rings
    static constexpr int OFF_DO = 0;
    static constexpr int OFF_ROWS = TILE;  // Q on its way to TMEM, at the end dQ on its way out
    static constexpr int OFF_K = 2 * TILE;
    static constexpr int OFF_V = OFF_K + NK * TILE;
    static constexpr int OFF_CTRL = OFF_V + NV * TILE;
    static constexpr int SMEM_BYTES = OFF_CTRL + 2048 + 1024;
    static_assert(SMEM_BYTES <= 232448, "too much shared memory");
};

struct DqCtrl {
    uint64_t k_full[3], k_empty[3], v_full[2], v_empty[2], tail_ready;
    uint64_t ready, s_full, s_free, dz_full, dz_free, dq_full, mma_done;
    uint32_t tmem_base;
    int abort_flag;
    float delta[128];
};
static_assert(sizeof(DqCtrl) <= 2048, "control block too large");

constexpr uint32_t kDqTmemQ = 0, kDqTmemDz = 64, kDqTmemS = 128, kDqTmemDp = 256, kDqTmemDq = 384;
constexpr int kDqRegsLaunch = 168, kDqRegsCtl = 80, kDqRegsSoft = 208;
constexpr int kDqRegsSplitTotal = 128 * (kDqRegsCtl + 2 * kDqRegsSoft);
static_assert(kDqRegsSplitTotal <= kBwdTcThreads * kDqRegsLaunch, "register split exceeds the launch allocation");

// Grid: row tiles (fastest), splits of the keys, B * Hkv.
template <int D>
__global__ void __launch_bounds__(kBwdTcThreads, 1) attn_dq_tc_kernel(const __grid_constant__ TcBwdArgs g) {
    using L = DqLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    DqCtrl* ctrl = reinterpret_cast<DqCtrl*>(smem + L::OFF_CTRL);
    volatile int* abort_flag = &ctrl->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    next_may_start();
    const int R = g.G * g.n;
    const int rtiles = (R + 127) / 128;
    const int r0 = static_cast<int>(blockIdx.x % rtiles) * 128;
    const int split = static_cast<int>(blockIdx.x / rtiles % g.qsplits);
    const int bh = static_cast<int>(blockIdx.x / rtiles / g.qsplits);
    const int b = bh / g.Hkv, hk = bh % g.Hkv;
    const int len = g.length(b);
    // This block's key tiles [t0, t0 + T).
    const int tiles = (len + 127) / 128;
    const int t0 = static_cast<int>(static_cast<long long>(tiles) * split / g.qsplits);
    const int T = static_cast<int>(static_cast<long long>(tiles) * (split + 1) / g.qsplits) - t0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < L::NK; ++s) {
            ptx::mbar_init(&ctrl->k_full[s], 1);
            ptx::mbar_init(&ctrl->k_empty[s], 1);
        }
        for (int s = 0; s < L::NV; ++s) {
            ptx::mbar_init(&ctrl->v_full[s], 1);
            ptx::mbar_init(&ctrl->v_empty[s], 1);
        }
        ptx::mbar_init(&ctrl->tail_ready, 1);
        ptx::mbar_init(&ctrl->ready, 8);
        ptx::mbar_init(&ctrl->s_full, 1);
        ptx::mbar_init(&ctrl->s_free, 8);
        ptx::mbar_init(&ctrl->dz_full, 8);
        ptx::mbar_init(&ctrl->dz_free, 1);
        ptx::mbar_init(&ctrl->dq_full, 1);
        ptx::mbar_init(&ctrl->mma_done, 1);
        ctrl->abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tensormap(&g.k);
        ptx::prefetch_tensormap(&g.v);
    }
    if (warp == 1) {
        ptx::tmem_alloc(&ctrl->tmem_base, 512);
        ptx::tmem_relinquish();
    }
    __syncwarp();  // one thread of some warps has been elsewhere; setmaxnreg wants whole warps
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = ctrl->tmem_base;
    const uint64_t lim = g.wait_ns, dlim = g.drain_ns;

    if (warp < 4) {
      ptx::regs_dec<kDqRegsCtl>();
      if (warp == 0) {
        // ------------------------------------------------------------ producer
        int nk = 0, nv = 0;
        for (int t = 0; t < T; ++t) {
            const int sk = t % L::NK, sv = t % L::NV;
            bool ok = mbar_wait(&ctrl->k_empty[sk], ((t / L::NK) & 1) ^ 1, abort_flag, lim, &g_lard_fault, kFaultBwdProducer);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(&ctrl->k_full[sk], L::TILE);
                for (int c = 0; c < L::KC; ++c)
                    tma_load_4d(smem + L::OFF_K + sk * L::TILE + c * 16384, &g.k, &ctrl->k_full[sk], c * 64, (t0 + t) * 128,
                                g.khead ? hk : 0, g.kbatch ? b : 0);
            }
            __syncwarp();
            ++nk;
            ok = mbar_wait(&ctrl->v_empty[sv], ((t / L::NV) & 1) ^ 1, abort_flag, lim, &g_lard_fault, kFaultBwdProducer);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(&ctrl->v_full[sv], L::TILE);
                for (int c = 0; c < L::KC; ++c)
                    tma_load_4d(smem + L::OFF_V + sv * L::TILE + c * 16384, &g.v, &ctrl->v_full[sv], c * 64, (t0 + t) * 128,
                                g.vhead ? hk : 0, g.vbatch ? b : 0);
            }
            __syncwarp();
            ++nv;
            if ((t0 + t) * 128 + 128 > len) {  // K rows past the end meet dZ = 0 in dQ: they must not be NaN
                ok = mbar_wait(&ctrl->k_full[sk], (t / L::NK) & 1, abort_flag, lim, &g_lard_fault, kFaultBwdProducer);
                if (!__all_sync(0xffffffffu, ok)) break;
                uint8_t* k = smem + L::OFF_K + sk * L::TILE;
                for (int e = (len - (t0 + t) * 128) * 8 + lane; e < 1024; e += 32)
                    for (int c = 0; c < L::KC; ++c)
                        *reinterpret_cast<uint4*>(k + c * 16384 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&ctrl->tail_ready);
            }
        }
        // Let every copy this warp started land before the block can exit.
        for (int s = 0; s < L::NK && s < nk; ++s) drain(&ctrl->k_full[s], ((nk - 1 - s) / L::NK) & 1, dlim);
        for (int s = 0; s < L::NV && s < nv; ++s) drain(&ctrl->v_full[s], ((nv - 1 - s) / L::NV) & 1, dlim);
      } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (one thread)
        if (lane == 0) {
            constexpr uint32_t kIdescS = ptx::idesc_bf16(128, 128, 0, 0);
            constexpr uint32_t kIdescDq = ptx::idesc_bf16(128, D, 0, 1);
            constexpr uint32_t kHi = ptx::sdesc_hi(1024);
            const uint32_t do_k = ptx::sdesc_lo(ptx::smem_u32(smem + L::OFF_DO), 16);
            const uint32_t k_k = ptx::sdesc_lo(ptx::smem_u32(smem + L::OFF_K), 16);
            const uint32_t k_mn = ptx::sdesc_lo(ptx::smem_u32(smem + L::OFF_K), 16384);
            const uint32_t v_k = ptx::sdesc_lo(ptx::smem_u32(smem + L::OFF_V), 16);
            constexpr uint32_t kStage = L::TILE >> 4;
            auto wait = [&](uint64_t* bar, int parity) {
                return mbar_wait(bar, parity, abort_flag, lim, &g_lard_fault, kFaultBwdMma);
            };
            int ks = 0, kp = 0, vs = 0, vp = 0;  // next stage of each ring and the parity of its round
            auto issue_s = [&](bool tail) {      // S = Q K^T, dP = dO V^T of the next key tile
                if (!wait(&ctrl->k_full[ks], kp) || (tail && !wait(&ctrl->tail_ready, 0))) return false;
                const uint32_t kd = k_k + ks * kStage;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    if (kk == 0) ptx::umma_ts<0>(tmem + kDqTmemS, tmem + kDqTmemQ, kd, kHi, kIdescS);
                    else ptx::umma_ts<1>(tmem + kDqTmemS, tmem + kDqTmemQ + kk * 8, kd + ptx::desc_step_k(kk), kHi, kIdescS);
                }
                if (!wait(&ctrl->v_full[vs], vp)) return false;
                const uint32_t vd = v_k + vs * kStage;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    if (kk == 0) ptx::umma_ss<0>(tmem + kDqTmemDp, do_k, vd, kHi, kIdescS);
                    else ptx::umma_ss<1>(tmem + kDqTmemDp, do_k + ptx::desc_step_k(kk), vd + ptx::desc_step_k(kk), kHi, kIdescS);
                }
                ptx::umma_commit(&ctrl->s_full);
                ptx::umma_commit(&ctrl->v_empty[vs]);
                if (++ks == L::NK) { ks = 0; kp ^= 1; }
                if (++vs == L::NV) { vs = 0; vp ^= 1; }
                return true;
            };
            const bool ragged = len % 128 != 0 && t0 + T == tiles;  // the last of these tiles is
            bool ok = T > 0 && wait(&ctrl->ready, 0);
            if (ok) {
                ptx::tc_fence_after();
                ok = issue_s(ragged && T == 1);
            }
            int kq = 0;  // stage of the tile whose dZ comes next
            for (int t = 0; ok && t < T; ++t) {
                if (t + 1 < T) {  // as soon as S and dP of tile t are in registers
                    if (!(ok = wait(&ctrl->s_free, t & 1))) break;
                    ptx::tc_fence_after();
                    if (!(ok = issue_s(ragged && t + 2 == T))) break;
                }
                if (!(ok = wait(&ctrl->dz_full, t & 1))) break;
                ptx::tc_fence_after();
                const uint32_t kd = k_mn + kq * kStage;
                umma_ts_acc(tmem + kDqTmemDq, tmem + kDqTmemDz, kd, kHi, kIdescDq, t > 0 ? 1u : 0u);
#pragma unroll
                for (int kk = 1; kk < 8; ++kk)
                    ptx::umma_ts<1>(tmem + kDqTmemDq, tmem + kDqTmemDz + kk * 8, kd + ptx::desc_step_mn(kk), kHi, kIdescDq);
                ptx::umma_commit(&ctrl->dz_free);
                ptx::umma_commit(&ctrl->k_empty[kq]);
                if (++kq == L::NK) kq = 0;
            }
            if (ok) ptx::umma_commit(&ctrl->dq_full);
            ptx::umma_commit(&ctrl->mma_done);
            drain(&ctrl->mma_done, 0, dlim);
        }
        __syncwarp();
      }
    } else {
        ptx::regs_inc<kDqRegsSoft>();
        // ------------------------------------------------------------ dZ
        const int q4 = warp & 3;
        const int half = (warp - 4) >> 2;  // 64-column half of every tile
        const int row = q4 * 32 + lane;
        const int r = r0 + row;
        const bool row_ok = r < R;
        const int head = hk * g.G + (row_ok ? r / g.n : 0), pos = row_ok ? r % g.n : 0;
        const size_t grow = static_cast<size_t>(bh) * R + (row_ok ? r : 0);
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
        // Prologue: Q and dO rows into shared memory, each warp half of its 32 rows;
        // delta; Q on into TMEM.
        const __nv_bfloat16* od = row_ok ? g.dout.row(b, head, pos) : nullptr;
        {
            const uint32_t q_area = ptx::smem_u32(smem + L::OFF_ROWS);
            rows_to_operand<D>(q_area, q4 * 32, row_ok ? g.q.row(b, head, pos) : nullptr, lane, 16 * half, 16 * half + 16);
            rows_to_operand<D>(ptx::smem_u32(smem + L::OFF_DO), q4 * 32, od, lane, 16 * half, 16 * half + 16);
            copy_commit();
            constexpr int kLanes = D / 8;
            const __nv_bfloat16* oo = row_ok ? g.out.row(b, head, pos) : nullptr;
            const __nv_bfloat16* orest = row_ok && g.rest.p ? g.rest.row(b, head, pos) : nullptr;
#pragma unroll 4
            for (int k = 16 * half; k < 16 * half + 16; k += 32 / kLanes) {
                const int x = k + lane / kLanes, u = lane % kLanes;
                const __nv_bfloat16 *pd = shfl_ptr(od, x), *po = shfl_ptr(oo, x), *pr = shfl_ptr(orest, x);
                float s = 0.f;
                if (pd) {
                    const uint4 d4 = __ldg(reinterpret_cast<const uint4*>(pd) + u), o4 = __ldg(reinterpret_cast<const uint4*>(po) + u);
                    uint4 r4 = make_uint4(0u, 0u, 0u, 0u);
                    if (pr) r4 = __ldg(reinterpret_cast<const uint4*>(pr) + u);
                    const uint32_t xs[4] = {d4.x, d4.y, d4.z, d4.w}, ys[4] = {o4.x, o4.y, o4.z, o4.w};
                    const uint32_t rs[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s = fmaf(__uint_as_float(xs[e] << 16), __uint_as_float(ys[e] << 16) + __uint_as_float(rs[e] << 16), s);
                        s = fmaf(__uint_as_float(xs[e] & 0xffff0000u),
                                 __uint_as_float(ys[e] & 0xffff0000u) + __uint_as_float(rs[e] & 0xffff0000u), s);
                    }
                }
#pragma unroll
                for (int e = kLanes / 2; e > 0; e >>= 1) s += __shfl_xor_sync(0xffffffffu, s, e);
                if (u == 0) {
                    ctrl->delta[q4 * 32 + x] = s;
                    if (pd && split == 0) g.delta[static_cast<size_t>(bh) * R + r0 + q4 * 32 + x] = s;
                }
            }
            copy_wait<0>();
            ptx::fence_proxy_async_smem();
            ptx::named_bar_sync(1, 256);  // both halves of the rows are there
            if (half == 0) {
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t w[32];
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w[4 * u]), "=r"(w[4 * u + 1]), "=r"(w[4 * u + 2]), "=r"(w[4 * u + 3])
                                     : "r"(q_area + c * 16384 + row * 128 + ((u ^ (row & 7)) << 4))
                                     : "memory");
                    __syncwarp();
                    ptx::tmem_st32(lane_base + kDqTmemQ + c * 32, w);
                }
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&ctrl->ready);
        }
        const float delta = ctrl->delta[row];
        const float nl2 = row_ok ? -g.lse[grow] * kLog2e : 0.f;
        const float2 cf2 = splat2(g.cfac), nl22 = splat2(nl2), nd2 = splat2(-delta);
        bool ok = true;
        for (int t = 0; t < T; ++t) {
            const int seen = row_ok ? len - (t0 + t) * 128 - half * 64 : 0;  // of this thread's 64 keys
            ok = mbar_wait(&ctrl->s_full, t & 1, abort_flag, lim, &g_lard_fault, kFaultBwdSoftmax);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            ptx::tc_fence_after();
            float z[2][32], dp[2][32];
            __syncwarp();
            ptx::tmem_ld32(lane_base + kDqTmemS + half * 64, z[0]);
            ptx::tmem_ld32(lane_base + kDqTmemS + half * 64 + 32, z[1]);
            ptx::tmem_ld32(lane_base + kDqTmemDp + half * 64, dp[0]);
            ptx::tmem_ld32(lane_base + kDqTmemDp + half * 64 + 32, dp[1]);
            ptx::tmem_ld_wait(z[0]);
            ptx::reg_dep(z[1]);
            ptx::reg_dep(dp[0]);
            ptx::reg_dep(dp[1]);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&ctrl->s_free);
            uint32_t pk[32];
#pragma unroll
            for (int k = 0; k < 64; k += 2) {
                const float2 u = fma2(make_float2(z[k >> 5][k & 31], z[k >> 5][(k & 31) + 1]), cf2, nl22);
                const float2 p = make_float2(ptx::ex2(u.x), ptx::ex2(u.y));
                float2 x = mul2(p, add2(make_float2(dp[k >> 5][k & 31], dp[k >> 5][(k & 31) + 1]), nd2));
                if (seen < 64) {
                    if (k >= seen) x.x = 0.f;
                    if (k + 1 >= seen) x.y = 0.f;
                }
                pk[k >> 1] = ptx::pack_bf16x2(x.x, x.y);
            }
            // dZ(t - 1) has been read by its product.
            ok = mbar_wait(&ctrl->dz_free, (t & 1) ^ 1, abort_flag, lim, &g_lard_fault, kFaultBwdSoftmax);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            ptx::tc_fence_after();
            __syncwarp();
            ptx::tmem_st32(lane_base + kDqTmemDz + half * 32, pk);
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&ctrl->dz_full);
        }
        if (ok && T > 0) {
            ok = mbar_wait(&ctrl->dq_full, 0, abort_flag, lim, &g_lard_fault, kFaultBwdEpilogue);
            ok = __all_sync(0xffffffffu, ok);
            ptx::tc_fence_after();
        }
        if (ok) {
            const uint32_t area = ptx::smem_u32(smem + L::OFF_ROWS) + (half * 4 + q4) * (L::TILE / 8);
#pragma unroll
            for (int c = 0; c < D / 2; c += 32) {
                float o[32];
                __syncwarp();
                if (T > 0) {
                    ptx::tmem_ld32(lane_base + kDqTmemDq + half * (D / 2) + c, o);
                    ptx::tmem_ld_wait(o);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0.f;
                }
                if (g.qsplits > 1)
                    fp32_rows_out<D / 4>(area, lane, o,
                                         row_ok ? g.part_q + (static_cast<size_t>(split) * g.B * g.Hkv * R + grow) * D +
                                                      half * (D / 2) + c
                                                : nullptr);
                else
                    stage_bf16<D>(area, lane, c / 8, o, g.tau);
            }
            if (g.qsplits == 1)
                staged_rows_out<D>(area, row_ok ? g.dq.row(b, head, pos) + half * (D / 2) : nullptr, lane);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------- dK, dV
constexpr int kUnit = 64;  // query rows of a unit

template <int D>
struct DkvLayout {
    static constexpr int KC = D / 64;
    static constexpr int TILE = KC * 16384;  // K or V
    static constexpr int UNIT = KC * 8192;   // 64 rows of Q or dO
    static constexpr int NS = D == 128 ? 4 : 6;
    static constexpr int OFF_K = 0;
    static constexpr int OFF_V = TILE;
    static constexpr int OFF_U = 2 * TILE;  // stage s: Q at OFF_U + 2 s UNIT, dO behind it
    static constexpr int OFF_CTRL = OFF_U + NS * 2 * UNIT;
    static constexpr int CTRL_BYTES = 4096;
    static constexpr int SMEM_BYTES = OFF_CTRL + CTRL_BYTES + 1024;
    static_assert(SMEM_BYTES <= 232448, "too much shared memory");
};

struct DkvCtrl {
    uint64_t kv_full, u_full[6], u_empty[6], st_full[6];
    uint64_t s_full[2], p_full[2];
    uint64_t acc_full, mma_done;
    uint32_t tmem_base;
    int abort_flag;
    alignas(16) float nlse2[6][kUnit];  // -LSE log2(e); -infinity for rows past the end
    alignas(16) float ndelta[6][kUnit];
};
static_assert(sizeof(DkvCtrl) <= 4096, "control block too large");

// Descriptor low-word step for K step kk of a 64-row, K-major unit (8 KB a 64-column chunk).
__host__ __device__ constexpr uint32_t desc_step_k64(int kk) { return (kk >> 2) * (8192 >> 4) + (kk & 3) * (32 >> 4); }

// It starts beside dQ's last blocks and needs their delta.  How long those take is not this
// kernel's affair, so every role waits for that kernel's end before its first bounded wait
// that something formed from delta has to end; K, V, the first units and the first
// two S^T and dP^T come before that.
// Grid: key tiles of m (fastest), splits of the rows, B * Hkv.
template <int D>
__global__ void __launch_bounds__(kBwdTcThreads, 1) attn_dkdv_tc_kernel(const __grid_constant__ TcBwdArgs g) {
    using L = DkvLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    DkvCtrl* ctrl = reinterpret_cast<DkvCtrl*>(smem + L::OFF_CTRL);
    volatile int* abort_flag = &ctrl->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ktiles = (g.m + 127) / 128;
    const int j0 = static_cast<int>(blockIdx.x % ktiles) * 128;
    const int split = static_cast<int>(blockIdx.x / ktiles % g.ksplits);
    const int bh = static_cast<int>(blockIdx.x / ktiles / g.ksplits);
    const int b = bh / g.Hkv, hk = bh % g.Hkv;
    const int len = g.length(b);
    // This block's units [u0, u0 + U), those of the group's heads in a row.
    const int upn = (g.n + kUnit - 1) / kUnit;  // units of a head
    const int units = j0 < len ? g.G * upn : 0;
    const int u0 = static_cast<int>(static_cast<long long>(units) * split / g.ksplits);
    const int U = static_cast<int>(static_cast<long long>(units) * (split + 1) / g.ksplits) - u0;
    if (g.qsplits > 1 || g.ksplits > 1) next_may_start();

    if (threadIdx.x == 0) {
        ptx::mbar_init(&ctrl->kv_full, 1);
        for (int s = 0; s < L::NS; ++s) {
            ptx::mbar_init(&ctrl->u_full[s], 1);
            ptx::mbar_init(&ctrl->u_empty[s], 1);
            ptx::mbar_init(&ctrl->st_full[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&ctrl->s_full[i], 1);
            ptx::mbar_init(&ctrl->p_full[i], 4);
        }
        ptx::mbar_init(&ctrl->acc_full, 1);
        ptx::mbar_init(&ctrl->mma_done, 1);
        ctrl->abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tensormap(&g.k);
        ptx::prefetch_tensormap(&g.v);
        ptx::prefetch_tensormap(&g.q64);
        ptx::prefetch_tensormap(&g.do64);
    }
    if (warp == 1) {
        ptx::tmem_alloc(&ctrl->tmem_base, 512);
        ptx::tmem_relinquish();
    }
    __syncwarp();  // one thread of some warps has been elsewhere; setmaxnreg wants whole warps
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = ctrl->tmem_base;
    const uint64_t lim = g.wait_ns, dlim = g.drain_ns;

    if (warp < 4) {
      ptx::regs_dec<kDqRegsCtl>();
      if (warp == 0 && U > 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            ptx::mbar_arrive_expect_tx(&ctrl->kv_full, 2 * L::TILE);
            for (int c = 0; c < L::KC; ++c) {
                tma_load_4d(smem + L::OFF_K + c * 16384, &g.k, &ctrl->kv_full, c * 64, j0, g.khead ? hk : 0, g.kbatch ? b : 0);
                tma_load_4d(smem + L::OFF_V + c * 16384, &g.v, &ctrl->kv_full, c * 64, j0, g.vhead ? hk : 0, g.vbatch ? b : 0);
            }
        }
        __syncwarp();
        int issued = 0;
        for (int u = 0; u < U; ++u) {
            const int s = u % L::NS;
            if (u == L::NS) wait_for_kernel_before();  // no stage is free again before delta is there
            const bool ok = mbar_wait(&ctrl->u_empty[s], ((u / L::NS) & 1) ^ 1, abort_flag, lim, &g_lard_fault,
                                           kFaultBwdProducer);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (lane == 0) {
                const int head = hk * g.G + (u0 + u) / upn, i0 = (u0 + u) % upn * kUnit;
                uint8_t* dst = smem + L::OFF_U + s * 2 * L::UNIT;
                ptx::mbar_arrive_expect_tx(&ctrl->u_full[s], 2 * L::UNIT);
                for (int c = 0; c < L::KC; ++c) {
                    tma_load_4d(dst + c * 8192, &g.q64, &ctrl->u_full[s], c * 64, i0, g.qhead ? head : 0, g.qbatch ? b : 0);
                    tma_load_4d(dst + L::UNIT + c * 8192, &g.do64, &ctrl->u_full[s], c * 64, i0, g.dohead ? head : 0, g.dobatch ? b : 0);
                }
            }
            __syncwarp();
            ++issued;
        }
        // Let every copy this warp started land before the block can exit.
        drain(&ctrl->kv_full, 0, dlim);
        for (int s = 0; s < L::NS && s < issued; ++s) drain(&ctrl->u_full[s], ((issued - 1 - s) / L::NS) & 1, dlim);
      } else if (warp == 2) {
        // ------------------------------------------------------------ row statistics of each unit
        wait_for_kernel_before();  // delta
        for (int u = 0; u < U; ++u) {
            const int s = u % L::NS;
            const bool ok = mbar_wait(&ctrl->u_empty[s], ((u / L::NS) & 1) ^ 1, abort_flag, lim, &g_lard_fault,
                                           kFaultBwdProducer);
            if (!__all_sync(0xffffffffu, ok)) break;
            const int i0 = (u0 + u) % upn * kUnit;
            const size_t at = (static_cast<size_t>(bh) * g.G + (u0 + u) / upn) * g.n + i0;
#pragma unroll
            for (int k = 0; k < kUnit; k += 32) {
                const bool in = i0 + k + lane < g.n;
                ctrl->nlse2[s][k + lane] = in ? -g.lse[at + k + lane] * kLog2e : -INFINITY;
                ctrl->ndelta[s][k + lane] = in ? -g.delta[at + k + lane] : 0.f;
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&ctrl->st_full[s]);
        }
      } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (one thread)
        if (lane == 0) {
            constexpr uint32_t kIdescS = ptx::idesc_bf16(128, kUnit, 0, 0);
            constexpr uint32_t kIdescAcc = ptx::idesc_bf16(128, D, 0, 1);
            constexpr uint32_t kHi = ptx::sdesc_hi(1024);
            const uint32_t k_k = ptx::sdesc_lo(ptx::smem_u32(smem + L::OFF_K), 16);
            const uint32_t v_k = ptx::sdesc_lo(ptx::smem_u32(smem + L::OFF_V), 16);
            const uint32_t u_k = ptx::sdesc_lo(ptx::smem_u32(smem + L::OFF_U), 16);
            const uint32_t u_mn = ptx::sdesc_lo(ptx::smem_u32(smem + L::OFF_U), 8192);
            constexpr uint32_t kQ = 2 * L::UNIT >> 4, kDo = L::UNIT >> 4;
            auto wait = [&](uint64_t* bar, int parity) {
                return mbar_wait(bar, parity, abort_flag, lim, &g_lard_fault, kFaultBwdMma);
            };
            int next = 0, np = 0;             // stage of the next unit and the parity of its round
            auto issue_s = [&](int stream) {  // S^T = K Q^T, dP^T = V dO^T of the next unit
                if (!wait(&ctrl->u_full[next], np)) return false;
                const uint32_t q = u_k + next * kQ, o = q + kDo;
                const uint32_t ts = tmem + 256 + stream * 64, tp = ts + 128;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    if (kk == 0) ptx::umma_ss<0>(ts, k_k, q, kHi, kIdescS);
                    else ptx::umma_ss<1>(ts, k_k + ptx::desc_step_k(kk), q + desc_step_k64(kk), kHi, kIdescS);
                }
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    if (kk == 0) ptx::umma_ss<0>(tp, v_k, o, kHi, kIdescS);
                    else ptx::umma_ss<1>(tp, v_k + ptx::desc_step_k(kk), o + desc_step_k64(kk), kHi, kIdescS);
                }
                ptx::umma_commit(&ctrl->s_full[stream]);
                if (++next == L::NS) { next = 0; np ^= 1; }
                return true;
            };
            bool ok = U > 0 && wait(&ctrl->kv_full, 0);
            for (int u = 0; ok && u < 2 && u < U; ++u) ok = issue_s(u);
            wait_for_kernel_before();  // P^T and dZ^T come after delta
            int s = 0;
            for (int u = 0; ok && u < U; ++u) {
                const int stream = u & 1;
                if (!(ok = wait(&ctrl->p_full[stream], (u >> 1) & 1))) break;
                ptx::tc_fence_after();
                const uint32_t q = u_mn + s * kQ, o = q + kDo;
                const uint32_t tp = tmem + 256 + stream * 64, tz = tp + 128;
                umma_ts_acc(tmem, tp, o, kHi, kIdescAcc, u > 0 ? 1u : 0u);
#pragma unroll
                for (int kk = 1; kk < kUnit / 16; ++kk) ptx::umma_ts<1>(tmem, tp + kk * 8, o + ptx::desc_step_mn(kk), kHi, kIdescAcc);
                umma_ts_acc(tmem + 128, tz, q, kHi, kIdescAcc, u > 0 ? 1u : 0u);
#pragma unroll
                for (int kk = 1; kk < kUnit / 16; ++kk)
                    ptx::umma_ts<1>(tmem + 128, tz + kk * 8, q + ptx::desc_step_mn(kk), kHi, kIdescAcc);
                ptx::umma_commit(&ctrl->u_empty[s]);
                if (++s == L::NS) s = 0;
                if (u + 2 < U) ok = issue_s(stream);  // behind the products that read P^T and dZ^T in its place
            }
            if (ok) ptx::umma_commit(&ctrl->acc_full);
            ptx::umma_commit(&ctrl->mma_done);
            drain(&ctrl->mma_done, 0, dlim);
        }
        __syncwarp();
      }
    } else {
        ptx::regs_inc<kDqRegsSoft>();
        // ------------------------------------------------------------ P^T, dZ^T
        const int q4 = warp & 3;
        const int i = (warp - 4) >> 2;  // units u with u & 1 == i
        const int key = j0 + q4 * 32 + lane;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
        const uint32_t ts = lane_base + 256 + i * 64, tp = ts + 128;
        const float2 cf2 = splat2(g.cfac);
        bool ok = true;
        wait_for_kernel_before();  // each unit's statistics come after delta
        for (int u = i; u < U; u += 2) {
            const int s = u % L::NS;
            ok = mbar_wait(&ctrl->st_full[s], (u / L::NS) & 1, abort_flag, lim, &g_lard_fault, kFaultBwdSoftmax) &&
                 mbar_wait(&ctrl->s_full[i], (u >> 1) & 1, abort_flag, lim, &g_lard_fault, kFaultBwdSoftmax);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            ptx::tc_fence_after();
            float z[2][32], dp[2][32];
            __syncwarp();
            ptx::tmem_ld32(ts, z[0]);
            ptx::tmem_ld32(ts + 32, z[1]);
            ptx::tmem_ld32(tp, dp[0]);
            ptx::tmem_ld32(tp + 32, dp[1]);
            ptx::tmem_ld_wait(z[0]);
            ptx::reg_dep(z[1]);
            ptx::reg_dep(dp[0]);
            ptx::reg_dep(dp[1]);
            const float4* nl = reinterpret_cast<const float4*>(ctrl->nlse2[s]);
            const float4* nd = reinterpret_cast<const float4*>(ctrl->ndelta[s]);
            uint32_t pk[32], zk[32];
#pragma unroll
            for (int k = 0; k < 64; k += 4) {
                const float4 l4 = nl[k >> 2], d4 = nd[k >> 2];
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const int c = k + e;
                    const float2 w = fma2(make_float2(z[c >> 5][c & 31], z[c >> 5][(c & 31) + 1]), cf2,
                                          e ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y));
                    const float2 p = make_float2(ptx::ex2(w.x), ptx::ex2(w.y));
                    const float2 x = mul2(p, add2(make_float2(dp[c >> 5][c & 31], dp[c >> 5][(c & 31) + 1]),
                                                  e ? make_float2(d4.z, d4.w) : make_float2(d4.x, d4.y)));
                    pk[c >> 1] = ptx::pack_bf16x2(p.x, p.y);
                    zk[c >> 1] = ptx::pack_bf16x2(x.x, x.y);
                }
            }
            __syncwarp();
            ptx::tmem_st32(ts, pk);
            ptx::tmem_st32(tp, zk);
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&ctrl->p_full[i]);
        }
        if (ok && U > 0) {
            ok = mbar_wait(&ctrl->acc_full, 0, abort_flag, lim, &g_lard_fault, kFaultBwdEpilogue);
            ok = __all_sync(0xffffffffu, ok);
            ptx::tc_fence_after();
        }
        if (ok) {  // warpgroup 0 writes dV, 1 dK; keys past the length get zeros
            // Through K's tile and V's, which the last S^T and dP^T have read.
            const uint32_t area = ptx::smem_u32(smem + (i ? L::OFF_K : L::OFF_V)) + q4 * (L::TILE / 4);
            const float scale = i ? g.tau : 1.f;
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                float o[32];
                __syncwarp();
                if (U > 0) {
                    ptx::tmem_ld32(lane_base + i * 128 + c, o);
                    ptx::tmem_ld_wait(o);
                }
                if (U == 0 || key >= len) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0.f;
                }
                if (g.ksplits > 1)
                    fp32_rows_out<32>(area, lane, o,
                                      key < g.m ? (i ? g.part_k : g.part_v) +
                                                      ((static_cast<size_t>(split) * g.B * g.Hkv + bh) * g.m + key) * D + c
                                                : nullptr);
                else
                    stage_bf16<D * 2>(area, lane, c / 8, o, scale);
            }
            if (g.ksplits == 1) staged_rows_out<D * 2>(area, key < g.m ? (i ? g.dk : g.dv).row(b, hk, key) : nullptr, lane);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(tmem, 512);
}

}  // namespace attn
}  // namespace lard
