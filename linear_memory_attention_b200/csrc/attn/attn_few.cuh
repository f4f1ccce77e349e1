// attn_few.cuh -- the forward pass of up to 16 query rows a key head (bf16):
// single tokens of grouped heads, short queries.
//
// Such a pass reads every key and value for a few multiply-adds: HBM bounds it,
// and what counts is bytes in flight (three blocks an SM, 64 KB of boxes each).
// Measured, 16 sequences x 8 key heads x 8000 keys at d = 128 (524 MB where all are
// used): 84 us, 6.2 TB/s; of ragged lengths, 378 MB, 72 us, 5.2 TB/s: the longest
// sequences' blocks end last.  Each warp takes groups of 16 keys on its
// own, which TMA brings into a queue of its own in shared memory (boxes of 16
// rows x 64 columns, 128-byte swizzle), and feeds them to m16n8k16 products;
// warps never wait for one another until the end.  The order of a product's
// inner index is free, so that every operand is a 16-byte piece, and pieces are
// chosen so that eight lanes in a row read different banks:
//   S = Q K^T   inner index d: lane 4 g + c takes pieces 2c, 2c + 1 of key g's 64-column
//               chunks, 8 elements that serve four k-pairs; Q's fragments
//               take the same order.
//   O += P V    inner index key: S's accumulators are P's A fragments as they are.
//               Output column n of product t stands for d = 64 (t / 8) + 8 n + t % 8,
//               so that a lane takes piece g of its four keys' chunks.
// (Single rows by untiled bulk copies stop at one copy per 16 cycles and SM; they and
// 16-byte copies by the threads reach 4.1 to 4.3 TB/s.)
// Rows' maxima, sums and O are per warp; a reference m rises only by steps above
// 2^8, as in the tensor-core pass.  The warps of a block are joined through
// shared memory, the blocks of a cluster (up to 8 share a problem's keys)
// through distributed shared memory, clusters by the join kernel.
#pragma once

#include <cooperative_groups.h>

#include "attn_common.cuh"
#include "attn_fwd_tc.cuh"
#include "attn_ptx.cuh"

namespace lard {
namespace attn {

struct FewArgs {
    TcSeg seg[2];  // boxes of 16 rows
    View<const __nv_bfloat16> q;
    View<__nv_bfloat16> out, rest;
    float* lse;
    int nseg, PB, Hkv, G, n, R;  // as in TcFwdArgs; R <= 16
    int cluster, splits;         // blocks of a cluster; clusters of a problem
    int split0, join;
    int second;  // the call's second pass, which runs beside the first
    long long rows;
    float* part_o;
    float* part_lse;
    float cfac;
    unsigned long long wait_ns, drain_ns;
};

constexpr int kFewRows = 16;
constexpr int kFewRise = 8;

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 shared16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

constexpr int kFewWarps = 4;

template <int D>
struct FewLayout {
    static constexpr int KI = D / 32;  // 16-byte pieces of a key that a lane takes
    static constexpr int NT = D / 8;   // output tiles
    static constexpr int KC = D / 64;  // 64-column chunks of a row, 2 KB each for 16 rows
    static constexpr int OFF_V = KC * 2048;
    static constexpr int STAGE = 2 * OFF_V;  // of a warp
    static constexpr int NS = D == 128 ? 2 : 4;
    static constexpr int QUEUE = kFewWarps * NS * STAGE;
    // At the end the warps' rows, and behind them the block's, take the queues' place.
    static constexpr int OFF_JOINED = kFewWarps * kFewRows * (D + 2) * 4;
    static_assert(OFF_JOINED + kFewRows * (D + 2) * 4 <= QUEUE, "no room for the join");
    static constexpr int OFF_BARS = QUEUE;
    static constexpr int SMEM_BYTES = QUEUE + kFewWarps * NS * 8 + 16 + 1024;
};

// Grid: the blocks of a cluster (fastest), problems, clusters along the keys.
template <int D>
__global__ void __launch_bounds__(32 * kFewWarps, 3) attn_few_kernel(const __grid_constant__ FewArgs g) {
    using L = FewLayout<D>;
    if (g.join) next_may_start();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* few_smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    constexpr int KI = L::KI, NT = L::NT;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gq = lane >> 2, c = lane & 3;
    const int rank = static_cast<int>(blockIdx.x % g.cluster);
    const int at = static_cast<int>(blockIdx.x / g.cluster);
    const int problems = g.PB * g.Hkv;
    const int ph = at % problems, split = at / problems;
    const int pb = ph / g.Hkv, hk = ph % g.Hkv;
    const int Gn = g.G * g.n;

    // The problem's groups of 16 keys, those of both segments in a row, are dealt
    // evenly to its blocks in runs, and within a block to the warps in turn.
    const int len0 = g.seg[0].length(pb), len1 = g.nseg > 1 ? g.seg[1].length(pb) : 0;
    const int groups0 = (len0 + 15) / 16, groups = groups0 + (len1 + 15) / 16;
    const int blocks = g.cluster * g.splits, block = split * g.cluster + rank;
    const int first = static_cast<int>(static_cast<long long>(groups) * block / blocks);
    const int end = static_cast<int>(static_cast<long long>(groups) * (block + 1) / blocks);
    auto global_row = [&](int r) { return (static_cast<long long>(pb + r / Gn) * g.Hkv + hk) * Gn + r % Gn; };

    uint64_t* bars = reinterpret_cast<uint64_t*>(few_smem + L::OFF_BARS) + warp * L::NS;
    int* abort_word = reinterpret_cast<int*>(few_smem + L::OFF_BARS + kFewWarps * L::NS * 8);
    volatile int* abort_flag = abort_word;
    if (lane == 0)
        for (int s = 0; s < L::NS; ++s) ptx::mbar_init(&bars[s], 1);
    if (threadIdx.x == 0) *abort_word = 0;
    ptx::fence_mbar_init();
    __syncthreads();
    uint8_t* queue = few_smem + warp * (L::NS * L::STAGE);
    auto fetch = [&](int grp, int stage) {  // one lane
        const bool second = grp >= groups0;
        const TcSeg& s = g.seg[second ? 1 : 0];
        const int j0 = (second ? grp - groups0 : grp) * 16;
        uint8_t* dst = queue + stage * L::STAGE;
        ptx::mbar_arrive_expect_tx(&bars[stage], L::STAGE);
        for (int u = 0; u < L::KC; ++u)
            tma_load_4d(dst + u * 2048, &s.k, &bars[stage], u * 64, j0, s.khead ? hk : 0, s.kbatch ? pb : 0);
        for (int u = 0; u < L::KC; ++u)
            tma_load_4d(dst + L::OFF_V + u * 2048, &s.v, &bars[stage], u * 64, j0, s.vhead ? hk : 0, s.vbatch ? pb : 0);
    };
    int next = first + warp, issued = 0;
    for (; issued < L::NS && next < end; ++issued, next += kFewWarps)
        if (lane == 0) fetch(next, issued);

    // Q fragments: rows gq and gq + 8.
    uint32_t qf[2 * KI][4];
    int pos[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = gq + 8 * h;
        const int b = pb + r / Gn, rem = r % Gn;
        pos[h] = rem % g.n;
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (r < g.R) x = *reinterpret_cast<const uint4*>(g.q.row(b, hk * g.G + rem / g.n, pos[h]) + ((i >> 1) * 8 + 2 * c + (i & 1)) * 8);
            qf[2 * i][h] = x.x;
            qf[2 * i][2 + h] = x.y;
            qf[2 * i + 1][h] = x.z;
            qf[2 * i + 1][2 + h] = x.w;
        }
    }
    float o[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][e] = 0.f;

    // Swizzled pieces: unit x of row r lies at r * 128 + ((x ^ (r & 7)) << 4).
    const uint32_t base_s = ptx::smem_u32(queue);
    const uint32_t kp[2] = {base_s + gq * 128 + (((2 * c) ^ gq) << 4), base_s + gq * 128 + (((2 * c + 1) ^ gq) << 4)};
    const uint32_t vp[2] = {base_s + L::OFF_V + 2 * c * 128 + ((gq ^ (2 * c)) << 4),
                            base_s + L::OFF_V + (2 * c + 1) * 128 + ((gq ^ (2 * c + 1)) << 4)};
    bool ok = true;
    int done = 0;
    for (int grp = first + warp; grp < end; grp += kFewWarps, ++done) {
        const int stage = done % L::NS;
        ok = ptx::mbar_wait(&bars[stage], (done / L::NS) & 1, abort_flag, g.wait_ns, &g_lard_fault, kFaultFwdProducer);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const uint32_t at_stage = stage * L::STAGE;
        const bool second = grp >= groups0;
        const TcSeg& s = g.seg[second ? 1 : 0];
        const int len = second ? len1 : len0, j0 = (second ? grp - groups0 : grp) * 16;
        const bool tail = j0 + 16 > len;
        if (tail) {  // values past the end meet P = 0: they must not be NaN
            for (int e = (len - j0) * 8 + lane; e < 128; e += 32)
                for (int u = 0; u < L::KC; ++u)
                    *reinterpret_cast<uint4*>(queue + at_stage + L::OFF_V + u * 2048 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
            __syncwarp();
        }
        float z[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}}, y[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int i = 0; i < KI; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t) {  // two chains a tile: a product waits for the one before it in its chain
                const uint4 k = shared16(kp[i & 1] + at_stage + (i >> 1) * 2048 + t * 1024);
                mma_16816(z[t], qf[2 * i], k.x, k.y);
                mma_16816(y[t], qf[2 * i + 1], k.z, k.w);
            }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[t][e] += y[t][e];
        // z[t][2 h + e]: row gq + 8 h, key j0 + 8 t + 2 c + e.
        float base[2];
        bool any_rise = false;
        float sc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (j0 + 16 > len - (s.causal ? g.n - 1 : 0)) {  // some row sees less than the whole group
                const int lim = (s.causal ? causal_limit(len, g.n, pos[h]) : len) - j0 - 2 * c;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (8 * t + e >= lim) z[t][2 * h + e] = -INFINITY;
            }
            float top = fmaxf(fmaxf(z[0][2 * h], z[0][2 * h + 1]), fmaxf(z[1][2 * h], z[1][2 * h + 1]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)) * g.cfac;
            const bool rise = top > m[h] + kFewRise;
            sc[h] = rise ? ptx::ex2(m[h] - top) : 1.f;
            if (rise) m[h] = top;
            any_rise = any_rise || rise;
            base[h] = m[h] == -INFINITY ? 0.f : m[h];  // nothing seen yet: every exponential below is 0
        }
        if (__any_sync(0xffffffffu, any_rise)) {
            l[0] *= sc[0];
            l[1] *= sc[1];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                o[t][0] *= sc[0];
                o[t][1] *= sc[0];
                o[t][2] *= sc[1];
                o[t][3] *= sc[1];
            }
        }
        uint32_t pf[4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float p0 = ptx::ex2(fmaf(z[t][2 * h], g.cfac, -base[h]));
                const float p1 = ptx::ex2(fmaf(z[t][2 * h + 1], g.cfac, -base[h]));
                l[h] += p0 + p1;
                pf[2 * t + h] = ptx::pack_bf16x2(p0, p1);
            }
#pragma unroll
        for (int u = 0; u < NT / 8; ++u) {
            uint32_t v[4][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint4 x = shared16(vp[e & 1] + at_stage + u * 2048 + (e >> 1) * 1024);
                v[e][0] = x.x;
                v[e][1] = x.y;
                v[e][2] = x.z;
                v[e][3] = x.w;
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                mma_16816(o[8 * u + 2 * w], pf, __byte_perm(v[0][w], v[1][w], 0x5410), __byte_perm(v[2][w], v[3][w], 0x5410));
                mma_16816(o[8 * u + 2 * w + 1], pf, __byte_perm(v[0][w], v[1][w], 0x7632), __byte_perm(v[2][w], v[3][w], 0x7632));
            }
        }
        if (tail) ptx::fence_proxy_async_smem();  // the zeros before the next copy into this stage
        __syncwarp();                             // every lane has its pieces
        if (next < end) {
            if (lane == 0) fetch(next, stage);
            ++issued;
            next += kFewWarps;
        }
    }
    // Let every copy that this warp requested land.
    for (; done < issued; ++done) drain(&bars[done % L::NS], (done / L::NS) & 1, g.drain_ns);
    // Join the warps.  o[t][2 h + e]: row gq + 8 h, d = 64 (t / 8) + 8 (2 c + e) + t % 8.
    float* so = reinterpret_cast<float*>(few_smem);  // [warps][16][D]
    float* sm = so + kFewWarps * kFewRows * D;       // [warps][16]
    float* sl = sm + kFewWarps * kFewRows;           // [warps][16]
    __syncthreads();  // the queues are empty
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        const int r = gq + 8 * h;
        if (c == 0) {
            sm[warp * kFewRows + r] = m[h];
            sl[warp * kFewRows + r] = l[h];
        }
        if (r < g.R) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int t = 0; t < NT; t += 4)
                    store4(so + (warp * kFewRows + r) * D + t / 8 * 64 + (2 * c + e) * 8 + t % 8,
                           make_float4(o[t][2 * h + e], o[t + 1][2 * h + e], o[t + 2][2 * h + e], o[t + 3][2 * h + e]));
        }
    }
    __syncthreads();
    float* jo = reinterpret_cast<float*>(few_smem + L::OFF_JOINED);  // [16][D], sums to the reference jm
    float* jm = jo + kFewRows * D;
    float* jl = jm + kFewRows;
    for (int e = threadIdx.x; e < g.R * (D / 4); e += 32 * kFewWarps) {
        const int r = e / (D / 4), x = e % (D / 4) * 4;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) top = fmaxf(top, sm[w * kFewRows + r]);
        const float ref = top == -INFINITY ? 0.f : top;
        float total = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
            const float f = ptx::ex2(sm[w * kFewRows + r] - ref);
            const float4 y = load4(so + (w * kFewRows + r) * D + x);
            total = fmaf(f, sl[w * kFewRows + r], total);
            acc = make_float4(fmaf(f, y.x, acc.x), fmaf(f, y.y, acc.y), fmaf(f, y.z, acc.z), fmaf(f, y.w, acc.w));
        }
        store4(jo + r * D + x, acc);
        if (x == 0) {
            jm[r] = top;
            jl[r] = total;
        }
    }
    // The blocks of a cluster write a share of the problem's rows each.
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    if (g.cluster > 1) cluster.sync();
    else __syncthreads();
    for (int e = rank * (32 * kFewWarps) + threadIdx.x; e < g.R * (D / 4); e += g.cluster * 32 * kFewWarps) {
        const int r = e / (D / 4), x = e % (D / 4) * 4;
        float top = -INFINITY;
        for (int w = 0; w < g.cluster; ++w) top = fmaxf(top, *cluster.map_shared_rank(jm + r, w));
        const float ref = top == -INFINITY ? 0.f : top;
        float total = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < g.cluster; ++w) {
            const float f = ptx::ex2(*cluster.map_shared_rank(jm + r, w) - ref);
            const float4 y = *reinterpret_cast<const float4*>(cluster.map_shared_rank(jo + r * D + x, w));
            total = fmaf(f, *cluster.map_shared_rank(jl + r, w), total);
            acc = make_float4(fmaf(f, y.x, acc.x), fmaf(f, y.y, acc.y), fmaf(f, y.z, acc.z), fmaf(f, y.w, acc.w));
        }
        const float inv = total == 0.f ? 0.f : 1.f / total;
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        const float lse = total == 0.f ? -INFINITY : (top + log2f(total)) * kLn2;
        const long long row = global_row(r);
        if (*abort_flag) continue;
        if (g.join) {
            const long long prow = (g.split0 + split) * g.rows + row;
            store4(g.part_o + prow * D + x, acc);
            if (x == 0) g.part_lse[prow] = lse;
        } else {
            const int b = pb + r / Gn, rem = r % Gn;
            store4(g.out.row(b, hk * g.G + rem / g.n, rem % g.n) + x, acc);
            if (g.rest.p)
                store4(g.rest.row(b, hk * g.G + rem / g.n, rem % g.n) + x,
                       make_float4(rounding_rest(acc.x), rounding_rest(acc.y), rounding_rest(acc.z), rounding_rest(acc.w)));
            if (x == 0) g.lse[row] = lse;
        }
    }
    if (g.cluster > 1) cluster.sync();       // no block leaves while another reads its rows
    if (g.second) wait_for_kernel_before();  // whoever waits for this pass has waited for the first
}

}  // namespace attn
}  // namespace lard
