// attn_fwd_tc.cuh -- the forward pass on the 5th-generation tensor cores (bf16).
//
// A stream owns 128 query rows and a run of key tiles; a block works on two, so
// that the tensor pipe has one stream's products while the other's exponentials
// are computed.  By rows (kByKeys = 0): stream i owns the rows of its own tile,
// and both read every key tile.  By keys (kByKeys = 1; at most 128 rows): both own the
// same rows, stream i the key tiles 2t + i, and the two are joined at the end.
// Per stream and key tile of KT (128; 64 at d = 64, where tensor memory then has room for two
// blocks an SM, and exponentials, not products, are the bound):
//   S = Q K^T      A = Q (shared memory, K-major), B = K (K-major)
//   P = 2^(S c - m), row sums in fp32, P rounded to bf16 over S's TMEM columns
//   O += P V       A = P (TMEM), B = V (MN-major), O in TMEM
// A row's reference m follows its maximum only when that has risen by more
// than 2^8: P then stays below 2^8 and in bf16's relative precision whatever
// m is, O and l are rescaled rarely, and the softmax threads do it themselves.
// What bounds it: a stream's chain of S, exponentials, P V per tile, of which two
// streams overlap.  At d = 128 a tile's products take 1024 cycles of the tensor pipe
// and its exponentials 1024 (128 x 128 / 16) of their unit; a step (a tile of each
// stream) takes about 3650: 1450 from a stream's P to its next S (products of both
// streams and some 340 cycles from the last product to who waits for it), 2100 for
// its softmax.  Measured, one B200: 4096 rows x 16384 keys, 32 heads over 8, d = 128: 0.88 ms
// and 47 us of joining, 1.25 PFLOP/s (alternated with other work; under the
// 1000 W cap 1.02 ms); 4 x 4096 x 4096, d = 64: 765 us, 718 TFLOP/s, where the
// exponential unit is the nearer bound (tiles of 64 keys and two blocks an SM: 20 %
// over tiles of 128 and one).
// A block's beginning and end take some 16000 cycles beside its steps: 2000 to set up (Q
// and the first K come meanwhile), 1500 to the first S, a first softmax 3000 longer than
// the others (instructions not cached yet), 900 for the last P V, 4000 to 5000 to write its rows, 1600
// between two blocks of an SM.
// Tried and slower at d = 128: four softmax warpgroups; part of the exponentials on
// the FMA pipe; units of 64 keys with two S a stream (1.25 ms); one stream a block
// and two blocks an SM (10 %).
// Key tiles past a sequence's length are never visited.  Values of rows past
// it inside the last tile are zeroed in shared memory before the product (0
// times what is there could be NaN); their logits are replaced by -infinity.
// TMEM: S of stream i at KT i, O in the upper half.
// Roles:
//   warp 0       TMA producer of the K / V ring
//   warp 1       TMEM owner, MMA issuer
//   warps 4 on   a warpgroup for each stream: Q rows into shared memory, softmax
//                (one row a thread), the epilogue
#pragma once

#include "../lard_exp2.cuh"
#include "attn_common.cuh"
#include "attn_ptx.cuh"

namespace lard {
namespace attn {

// Where a key segment lies for the TMA loads: maps {d, rows, heads, batch}.
struct TcSeg {
    CUtensorMap k, v;
    const int* len;
    int cap, causal;
    int khead, kbatch, vhead, vbatch;  // 1, or 0 where one block is shared (stride 0)
    __device__ __forceinline__ int length(int b) const {
        if (!len) return cap;
        const int l = len[b];
        return l < 0 ? 0 : (l > cap ? cap : l);
    }
};

// A launch; its fields are those of FwdArgs.
struct TcFwdArgs {
    TcSeg seg[2];
    View<const __nv_bfloat16> q;
    View<__nv_bfloat16> out, rest;
    float* lse;  // [B, Hq, n]
    int nseg, PB, Hkv, G, n, R;
    int splits, split0;  // with join: partial rows go to split0 + split
    int join;
    int second;  // the call's second pass, which runs beside the first
    long long rows;  // B Hkv G n
    float* part_o;
    float* part_lse;
    float cfac;
    unsigned long long wait_ns, drain_ns;
};

template <int D, int kByKeys>
struct FwdTcLayout {
    static constexpr int KT = D == 64 ? 64 : 128;  // keys of a tile
    static constexpr int KC = D / 64;
    static constexpr int TILE = KC * 16384;     // 128 rows of Q
    static constexpr int KV_TILE = KC * KT * 128;  // a K or V tile
    static constexpr int BLOCKS_PER_SM = D == 64 ? 2 : 1;
    static constexpr int NS = D == 64 ? 8 : (kByKeys ? 6 : 5);
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_KV = (kByKeys ? 1 : 2) * TILE;
    static constexpr int OFF_CTRL = OFF_KV + NS * KV_TILE;
    static constexpr int SMEM_BYTES = OFF_CTRL + 2048 + 1024;
    // By keys, the join stages a stream's O in the ring: 128 x D fp32.
    static_assert(!kByKeys || NS * KV_TILE >= 128 * (D + 4) * 4, "no room for the join");
    static_assert(BLOCKS_PER_SM * (SMEM_BYTES + 1024) <= 233472, "too much shared memory");
    // Tensor memory: S of stream i at KT i, O at TMEM_O + TMEM_O_STEP i.
    static constexpr int TMEM_COLS = 512 / BLOCKS_PER_SM, TMEM_O = TMEM_COLS / 2, TMEM_O_STEP = TMEM_COLS / 4;
    static_assert(2 * KT <= TMEM_O && D <= TMEM_O_STEP, "too much tensor memory");
    // Registers a thread, and how the warpgroups share them.
    static constexpr int REGS_LAUNCH = D == 64 ? 80 : 168, REGS_CTL = D == 64 ? 32 : 80, REGS_SOFT = D == 64 ? 104 : 208;
    static constexpr int REGS_SPLIT = 128 * (REGS_CTL + 2 * REGS_SOFT);
    static_assert(REGS_SPLIT <= 384 * REGS_LAUNCH, "register split exceeds the launch allocation");
};
constexpr int kFwdTcThreads = 384;

struct FwdTcCtrl {
    uint64_t kv_full[8], kv_empty[8];
    uint64_t q_ready, mma_done;
    uint64_t tail_ready[2];  // of either segment: the producer may be a tail ahead of the issuer
    uint64_t s_full[2], p_full[2], o_full[2];
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(FwdTcCtrl) <= 2048, "control block too large");

constexpr float kRiseLog2 = 8.0f;

// Grid: row tiles (fastest), then splits, then PB * Hkv.
template <int D, int kByKeys>
__global__ void __launch_bounds__(kFwdTcThreads, (FwdTcLayout<D, kByKeys>::BLOCKS_PER_SM))
    attn_fwd_tc_kernel(const __grid_constant__ TcFwdArgs g) {
    using L = FwdTcLayout<D, kByKeys>;
    constexpr int KT = L::KT;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    FwdTcCtrl* ctrl = reinterpret_cast<FwdTcCtrl*>(smem + L::OFF_CTRL);
    volatile int* abort_flag = &ctrl->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (g.join) next_may_start();

    constexpr int kRowsPerBlock = kByKeys ? 128 : 256;
    const int rtiles = (g.R + kRowsPerBlock - 1) / kRowsPerBlock;
    const int r0 = static_cast<int>(blockIdx.x % rtiles) * kRowsPerBlock;
    const int split = static_cast<int>(blockIdx.x / rtiles % g.splits);
    const int ph = static_cast<int>(blockIdx.x / rtiles / g.splits);
    const int pb = ph / g.Hkv, hk = ph % g.Hkv;

    // This block's key tiles [t0, t0 + T) of the segments' tiles in a row.
    const int len0 = g.seg[0].length(pb), len1 = g.nseg > 1 ? g.seg[1].length(pb) : 0;
    const int tiles0 = (len0 + KT - 1) / KT;
    int t0, T;
    {
        const long long all = static_cast<long long>(tiles0) + (len1 + KT - 1) / KT;
        t0 = static_cast<int>(all * split / g.splits);
        T = static_cast<int>(all * (split + 1) / g.splits) - t0;
    }
    // Streams and their steps: by rows each step is one tile for both, by keys two tiles.
    const int nstream = kByKeys ? 2 : (g.R - r0 > 128 ? 2 : 1);
    auto steps = [&](int i) { return kByKeys ? (T + 1 - i) / 2 : (i < nstream ? T : 0); };
    const int S = steps(0);
    auto tile_of = [&](int t, int i) { return t0 + (kByKeys ? 2 * t + i : t); };
    // Segment and first key of a tile.
    auto seg_of = [&](int tile) { return tile < tiles0 ? 0 : 1; };
    auto key_of = [&](int tile) { return (tile < tiles0 ? tile : tile - tiles0) * KT; };
    auto is_tail = [&](int tile) { return (tile < tiles0 ? len0 : len1) - key_of(tile) < KT; };
    constexpr int kTiles = kByKeys ? 2 : 1;  // K (and V) tiles of a step
    // The row of a softmax thread: stream i, row `row` of its tile.
    struct Row {
        bool in;
        int b, head, pos, rem;
    };
    auto row_of = [&](int i, int row) {
        const int Gn = g.G * g.n, r = r0 + (kByKeys ? 0 : i * 128) + row;
        Row x;
        x.in = r < g.R;
        x.b = pb + (x.in ? r / Gn : 0);
        x.rem = x.in ? r % Gn : 0;
        x.head = hk * g.G + x.rem / g.n;
        x.pos = x.rem % g.n;
        return x;
    };
    auto load_tile = [&](int slot, int tile, bool is_v) {  // one thread
        const TcSeg& seg = g.seg[seg_of(tile)];
        uint8_t* dst = smem + L::OFF_KV + slot * L::KV_TILE;
        ptx::mbar_arrive_expect_tx(&ctrl->kv_full[slot], L::KV_TILE);
        for (int c = 0; c < L::KC; ++c)
            tma_load_4d(dst + c * KT * 128, is_v ? &seg.v : &seg.k, &ctrl->kv_full[slot], c * 64, key_of(tile),
                        (is_v ? seg.vhead : seg.khead) ? hk : 0, (is_v ? seg.vbatch : seg.kbatch) ? pb : 0);
    };

    // What the first products read is requested before all else (it takes as long as the
    // rest of the set-up): Q, rows past the end as zeros (by keys the two streams share
    // one tile and the work), and the first step's K.
    const int primed = S == 0 ? 0 : (kByKeys && steps(1) > 0 ? 2 : 1);
    if (warp >= 4) {
        const int q4 = warp & 3, i = (warp - 4) >> 2;
        const Row x = row_of(i, q4 * 32 + lane);
        rows_to_operand<D>(ptx::smem_u32(smem + L::OFF_Q) + (kByKeys ? 0 : i * L::TILE), q4 * 32,
                           x.in ? g.q.row(x.b, x.head, x.pos) : nullptr, lane, kByKeys ? 16 * i : 0, kByKeys ? 16 * i + 16 : 32);
        copy_commit();
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::NS; ++s) {
            ptx::mbar_init(&ctrl->kv_full[s], 1);
            ptx::mbar_init(&ctrl->kv_empty[s], 1);
        }
        ptx::mbar_init(&ctrl->q_ready, 8);
        ptx::mbar_init(&ctrl->mma_done, 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&ctrl->tail_ready[i], 1);
            ptx::mbar_init(&ctrl->s_full[i], 1);
            ptx::mbar_init(&ctrl->p_full[i], 4);
            ptx::mbar_init(&ctrl->o_full[i], 1);
        }
        ctrl->abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
        for (int i = 0; i < primed; ++i) load_tile(i, tile_of(0, i), false);
    }
    if (warp == 3 && lane == 0)
        for (int s = 0; s < g.nseg; ++s) {
            ptx::prefetch_tensormap(&g.seg[s].k);
            ptx::prefetch_tensormap(&g.seg[s].v);
        }
    if (warp == 1) {
        ptx::tmem_alloc(&ctrl->tmem_base, L::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    __syncwarp();  // one thread of some warps has been elsewhere; setmaxnreg wants whole warps
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = ctrl->tmem_base;
    const uint64_t lim = g.wait_ns, dlim = g.drain_ns;

    if (warp < 4) {
      ptx::regs_dec<L::REGS_CTL>();
      if (warp == 0) {
        // ------------------------------------------------------------ producer
        // Ring order: the K tiles of step 0, its V tiles, the K tiles of step 1, ...
        int slot = 0, round = 0, issued = 0;  // units of the ring, the primed ones among them
        bool ok = true;
        for (int t = 0; ok && t < S; ++t) {
            for (int u = 0; ok && u < 2 * kTiles; ++u) {
                const int i = u % kTiles;
                const bool is_v = u >= kTiles;
                if (kByKeys && t >= steps(i)) continue;
                if (issued >= primed) {  // else requested already, and by now perhaps even released again
                    ok = mbar_wait(&ctrl->kv_empty[slot], (round & 1) ^ 1, abort_flag, lim, &g_lard_fault,
                                   kFaultFwdProducer);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) load_tile(slot, tile_of(t, i), is_v);
                    __syncwarp();
                }
                ++issued;
                if (is_v && is_tail(tile_of(t, i))) {  // values past the sequence's end: zeros
                    const int tile = tile_of(t, i);
                    ok = mbar_wait(&ctrl->kv_full[slot], round & 1, abort_flag, lim, &g_lard_fault, kFaultFwdProducer);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    uint8_t* v = smem + L::OFF_KV + slot * L::KV_TILE;
                    for (int e = ((seg_of(tile) ? len1 : len0) - key_of(tile)) * 8 + lane; e < KT * 8; e += 32)
                        for (int c = 0; c < L::KC; ++c)
                            *reinterpret_cast<uint4*>(v + c * KT * 128 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&ctrl->tail_ready[seg_of(tile)]);
                }
                if (++slot == L::NS) { slot = 0; ++round; }
            }
        }
        // Let every copy this warp started land before the block can exit.
        for (int s = 0; s < L::NS && s < issued; ++s) {
            const int last = s + L::NS * ((issued - 1 - s) / L::NS);
            drain(&ctrl->kv_full[s], (last / L::NS) & 1, dlim);
        }
      } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        // One thread, and little else in its loop than waits and products: what
        // it does between them, the tensor pipe waits for.
        if (lane == 0) {
            constexpr uint32_t kIdescS = ptx::idesc_bf16(128, KT, 0, 0);
            constexpr uint32_t kIdescO = ptx::idesc_bf16(128, D, 0, 1);
            constexpr uint32_t kHi = ptx::sdesc_hi(1024);
            const uint32_t q_lo = ptx::sdesc_lo(ptx::smem_u32(smem + L::OFF_Q), 16);
            const uint32_t kv_k = ptx::sdesc_lo(ptx::smem_u32(smem + L::OFF_KV), 16);
            const uint32_t kv_mn = ptx::sdesc_lo(ptx::smem_u32(smem + L::OFF_KV), 16384);
            // A place in the ring and the parity of its round.
            struct Place {
                int slot, parity;
                __device__ __forceinline__ void advance(int n) {
                    slot += n;
                    if (slot >= L::NS) {
                        slot -= L::NS;
                        parity ^= 1;
                    }
                }
            };
            auto wait = [&](uint64_t* bar, int parity) {
                return mbar_wait(bar, parity, abort_flag, lim, &g_lard_fault, kFaultFwdMma);
            };
            auto wait_place = [&](const Place& x) { return wait(&ctrl->kv_full[x.slot], x.parity); };
            auto release = [&](const Place& x) { ptx::umma_commit(&ctrl->kv_empty[x.slot]); };
            auto issue_s = [&](int i, const Place& x) {  // S_i = Q_i K^T; Q is one tile by keys
                const uint32_t a = q_lo + (kByKeys ? 0 : i * (L::TILE >> 4));
                const uint32_t b = kv_k + x.slot * (L::KV_TILE >> 4);
                const uint32_t d = tmem + i * KT;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    if (kk == 0) ptx::umma_ss<0>(d, a, b, kHi, kIdescS);
                    else ptx::umma_ss<1>(d, a + ptx::desc_step_k(kk), b + ptx::desc_step_k(kk), kHi, kIdescS);
                }
                ptx::umma_commit(&ctrl->s_full[i]);
            };
            auto issue_o = [&](int i, const Place& x, bool first) {  // O_i (+)= P_i V
                const uint32_t a = tmem + i * KT, b = kv_mn + x.slot * (L::KV_TILE >> 4);
                const uint32_t d = tmem + L::TMEM_O + i * L::TMEM_O_STEP;
                umma_ts_acc(d, a, b, kHi, kIdescO, first ? 0u : 1u);
#pragma unroll
                for (int kk = 1; kk < KT / 16; ++kk) ptx::umma_ts<1>(d, a + kk * 8, b + ptx::desc_step_mn(kk), kHi, kIdescO);
                ptx::umma_commit(&ctrl->o_full[i]);
            };
            // Ring order: step by step the K tiles, then the V tiles; by keys an
            // odd last step has one of each.
            Place k[2] = {{0, 0}, {kByKeys ? 1 : 0, 0}}, v[2] = {{kTiles, 0}, {2 * kTiles - 1, 0}};
            const int steps1 = steps(1);
            bool ok = S > 0 && wait(&ctrl->q_ready, 0);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (!ok || (i == 1 && steps1 == 0)) break;
                if (kByKeys || i == 0) ok = wait_place(k[i]);
                if (!ok) break;
                issue_s(i, k[i]);
                if (kByKeys || i == nstream - 1) release(k[i]);
            }
            for (int t = 0; ok && t < S; ++t) {
                const bool both = t < steps1;                  // stream 1 takes part in this step,
                const bool more0 = t + 1 < S, more1 = t + 1 < steps1;  // and either in the next
                if (kByKeys && !both) {
                    v[0] = k[0];
                    v[0].advance(1);
                }
                Place kn[2] = {k[0], k[1]};
                kn[0].advance(2 * kTiles);
                if (kByKeys) kn[1].advance(2 * kTiles);
                else kn[1] = kn[0];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (i == 1 && !both) continue;
                    const bool last = kByKeys || i == 1 || !both;  // stream to use a tile
                    if (kByKeys || i == 0) {
                        ok = ok && wait_place(v[i]);
                        // Rows past a sequence's end: the producer makes them zeros.
                        if (ok && is_tail(tile_of(t, i))) ok = wait(&ctrl->tail_ready[seg_of(tile_of(t, i))], 0);
                    }
                    ok = ok && wait(&ctrl->p_full[i], t & 1);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    issue_o(i, v[kByKeys ? i : 0], t == 0);
                    if (last) release(v[kByKeys ? i : 0]);
                    if (i == 0 ? more0 : more1) {  // behind the product that reads P where this S goes
                        if (kByKeys || i == 0) ok = wait_place(kn[i]);
                        if (!ok) break;
                        issue_s(i, kn[i]);
                        if (last) release(kn[i]);
                    }
                }
                k[0] = kn[0];
                k[1] = kn[1];
                v[0].advance(2 * kTiles);
                if (kByKeys) v[1].advance(2 * kTiles);
            }
            ptx::umma_commit(&ctrl->mma_done);
            drain(&ctrl->mma_done, 0, dlim);
        }
        __syncwarp();
      }
    } else {
        ptx::regs_inc<L::REGS_SOFT>();
        // ------------------------------------------------------------ softmax
        const int q4 = warp & 3;
        const int i = (warp - 4) >> 2;  // stream
        const int row = q4 * 32 + lane;
        copy_wait<0>();
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&ctrl->q_ready);
        const Row x = row_of(i, row);
        const bool row_ok = x.in;
        const int b = x.b, head = x.head, pos = x.pos;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
        const uint32_t ts = lane_base + i * KT, to = lane_base + L::TMEM_O + i * L::TMEM_O_STEP;
        const float cf = g.cfac;
        float m = -INFINITY, l = 0.f;  // reference (log2 domain) and sum of 2^(z - m)
        const int mine = steps(i);
        bool ok = true;
        for (int t = 0; t < mine; ++t) {
            const int tile = tile_of(t, i), s = seg_of(tile), j0 = key_of(tile);
            const int size = s ? len1 : len0;
            const int lim_keys = (g.seg[s].causal ? causal_limit(size, g.n, pos) : size) - j0;
            ok = mbar_wait(&ctrl->s_full[i], t & 1, abort_flag, lim, &g_lard_fault, kFaultFwdSoftmax);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            float z[KT / 32][32];
            __syncwarp();
#pragma unroll
            for (int c = 0; c < KT / 32; ++c) ptx::tmem_ld32(ts + c * 32, z[c]);
            ptx::tmem_ld_wait(z[0]);
#pragma unroll
            for (int c = 1; c < KT / 32; ++c) ptx::reg_dep(z[c]);
            if (lim_keys < KT) {
#pragma unroll
                for (int c = 0; c < KT; ++c)
                    if (c >= lim_keys) z[c >> 5][c & 31] = -INFINITY;
            }
            float top[4];  // of four runs of columns, side by side
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                constexpr int kRun = KT / 4;
                top[c] = fmaxf(z[c * kRun >> 5][c * kRun & 31], z[c * kRun >> 5][(c * kRun & 31) + 1]);
#pragma unroll
                for (int k = c * kRun + 2; k < (c + 1) * kRun; k += 2) top[c] = ptx::fmax3(top[c], z[k >> 5][k & 31], z[k >> 5][(k & 31) + 1]);
            }
            const float mx = fmaxf(ptx::fmax3(top[0], top[1], top[2]), top[3]) * cf;
            const bool rise = mx > m + kRiseLog2;  // always where the row has seen nothing yet and now does
            const float mnew = rise ? mx : m;
            if (__any_sync(0xffffffffu, rise) && t > 0) {
                // O(t - 1) is complete; bring it to the new reference.
                const float sc = rise ? ptx::ex2(m - mnew) : 1.f;
                l *= sc;
                ok = mbar_wait(&ctrl->o_full[i], (t - 1) & 1, abort_flag, lim, &g_lard_fault, kFaultFwdSoftmax);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ptx::tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    __syncwarp();
                    ptx::tmem_ld32(to + c, o);
                    ptx::tmem_ld_wait(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] *= sc;
                    ptx::tmem_st32(to + c, reinterpret_cast<const uint32_t(&)[32]>(o));
                    ptx::tmem_st_wait();
                }
            }
            m = mnew;
            const float base = m == -INFINITY ? 0.f : m;  // nothing seen yet: every exponential below is 0
            const float2 cf2 = splat2(cf), nb2 = splat2(-base);
            float2 sum = splat2(0.f);
#pragma unroll
            for (int h = 0; h < KT / 64; ++h) {
                uint32_t pk[32];
#pragma unroll
                for (int k = 0; k < 64; k += 2) {
                    const int c = h * 64 + k;
                    const float2 u = fma2(make_float2(z[c >> 5][c & 31], z[c >> 5][(c & 31) + 1]), cf2, nb2);
                    const float2 p = make_float2(ptx::ex2(u.x), ptx::ex2(u.y));
                    sum = add2(sum, p);
                    pk[k >> 1] = ptx::pack_bf16x2(p.x, p.y);
                }
                __syncwarp();
                ptx::tmem_st32(ts + h * 32, pk);
            }
            ptx::tmem_st_wait();
            l += sum.x + sum.y;
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&ctrl->p_full[i]);
        }
        // ------------------------------------------------------------ epilogue
        if (ok && mine > 0) {
            ok = mbar_wait(&ctrl->o_full[i], (mine - 1) & 1, abort_flag, lim, &g_lard_fault, kFaultFwdSoftmax);
            ok = __all_sync(0xffffffffu, ok);
            ptx::tc_fence_after();
        }
        float* stage = reinterpret_cast<float*>(smem + L::OFF_KV);  // [D][128], the ring is empty by then
        float* stats = stage + D * 128;                              // [stream][m, l][128]
        float w0 = 1.f, w1 = 0.f, m_all = m, l_all = l;
        if (kByKeys) {
            // Each stream leaves half of its columns and brings the other half home,
            // joined.  Its last product has read the ring for the last time, and
            // either waits for the other's at the first barrier.
            ptx::named_bar_sync(1, 256);
            stats[256 * i + row] = m;
            stats[256 * i + 128 + row] = l;
            if (ok && mine > 0) {
#pragma unroll 1
                for (int c = 0; c < D / 2; c += 32) {
                    const int col = (1 - i) * (D / 2) + c;
                    float o[32];
                    __syncwarp();
                    ptx::tmem_ld32(to + col, o);
                    ptx::tmem_ld_wait(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) stage[(col + k) * 128 + row] = o[k];
                }
            }
            ptx::named_bar_sync(1, 256);
            const float m1 = stats[256 * (1 - i) + row];
            m_all = fmaxf(m, m1);
            const float base = m_all == -INFINITY ? 0.f : m_all;
            w0 = ptx::ex2(m - base);
            w1 = ptx::ex2(m1 - base);
            l_all = l * w0 + stats[256 * (1 - i) + 128 + row] * w1;
        }
        // With no key nothing has waited for the stream's Q, whose place the rows below take.
        if (!kByKeys && mine == 0) ptx::named_bar_sync(1 + i, 128);
        if (ok && !*abort_flag) {
            const float inv = l_all == 0.f ? 0.f : 1.f / l_all;
            w0 *= inv;
            w1 *= inv;
            const float lse = l_all == 0.f ? -INFINITY : (m_all + log2f(l_all)) * kLn2;
            const long long grow = (static_cast<long long>(b) * g.Hkv + hk) * g.G * g.n + x.rem;
            const long long prow = (g.split0 + split) * g.rows + grow;
            const bool other = kByKeys && steps(1 - i) > 0;
            // This thread's columns [col0, col0 + kCols), through the warp's share of Q's
            // tile, which the last S has read, to memory.
            constexpr int kCols = kByKeys ? D / 2 : D, kPart = kByKeys ? D / 4 : 32;
            const int col0 = kByKeys ? i * (D / 2) : 0;
            const uint32_t area = ptx::smem_u32(smem + L::OFF_Q) + (kByKeys ? (4 * i + q4) * (L::TILE / 8) : i * L::TILE + q4 * (L::TILE / 4));
            __nv_bfloat16* out = row_ok && !g.join ? g.out.row(b, head, pos) : nullptr;
            __nv_bfloat16* rest = row_ok && !g.join && g.rest.p ? g.rest.row(b, head, pos) : nullptr;
            // A loop that is not unrolled: short calls wait for instructions here.
#pragma unroll 1
            for (int c = col0; c < col0 + kCols; c += 32) {
                float o[32];
                __syncwarp();
                if (mine > 0) {
                    ptx::tmem_ld32(to + c, o);
                    ptx::tmem_ld_wait(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] *= w0;
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0.f;
                }
                if (other) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = fmaf(stage[(c + k) * 128 + row], w1, o[k]);
                }
                if (g.join) {
                    fp32_rows_out<kPart>(area, lane, o, row_ok ? g.part_o + prow * D + c : nullptr);
                    continue;
                }
                stage_bf16<64>(area, lane, 0, o, 1.f);
                staged_rows_out<64>(area, row_ok ? out + c : nullptr, lane);
                if (g.rest.p) {
                    leave_rest(o);
                    stage_bf16<64>(area, lane, 0, o, 1.f);
                    staged_rows_out<64>(area, row_ok ? rest + c : nullptr, lane);
                }
            }
            if (row_ok && (!kByKeys || i == 0)) {
                if (g.join) g.part_lse[prow] = lse;
                else g.lse[grow] = lse;
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(tmem, L::TMEM_COLS);
    if (g.second) wait_for_kernel_before();  // whoever waits for this pass has waited for the first
}

}  // namespace attn
}  // namespace lard
