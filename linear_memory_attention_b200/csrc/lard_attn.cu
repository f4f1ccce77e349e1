// lard_attn.cu -- the C ABI of liblard_attn (declared in include/lard_attn.h):
// argument checks, per-device setup and kernel launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>
#include <utility>

#include "lard_attn.h"
#include "lard_host.h"
#include "lard_kernel_common.cuh"
#include "attn/attn_bwd_tc.cuh"
#include "attn/attn_common.cuh"
#include "attn/attn_few.cuh"
#include "attn/attn_fwd_tc.cuh"
#include "attn/attn_join.cuh"
#include "attn/attn_simt.cuh"

namespace {

using lard::attn::FwdArgs;
using lard::attn::KeySeg;
using lard::attn::View;
using bf16 = __nv_bfloat16;

constexpr unsigned long long kWaitLimitNs = 2000000000ull;   // 2 s per wait
constexpr unsigned long long kDrainLimitNs = 8000000000ull;  // 8 s per drain on the way out
constexpr int kMaxDevices = 64;
constexpr int kSms = 148;  // of a B200: plans depend on sizes alone, so that a workspace can be sized without a GPU
constexpr int kMaxRows = INT_MAX - 255;

std::mutex g_mu;
bool g_ready[kMaxDevices];
lard_status g_dev_status[kMaxDevices];
EncodeTiledFn g_encode = nullptr;

// One-time setup of device `dev` (made current by the caller).
lard_status setup_device(int dev) {
    std::lock_guard<std::mutex> lk(g_mu);
    if (dev < 0 || dev >= kMaxDevices) return LARD_ERR_UNSUPPORTED;
    if (g_ready[dev]) return g_dev_status[dev];
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return LARD_ERR_CUDA;
    lard_status st = LARD_OK;
    if (major != 10 || minor != 0) st = LARD_ERR_UNSUPPORTED;  // built for sm_100a only
    if (st == LARD_OK && !g_encode) {
        g_encode = find_encode_tiled();
        if (!g_encode) st = LARD_ERR_CUDA;
    }
    if (st == LARD_OK) {
        using namespace lard::attn;
        bool ok = true, fits = true;
        auto tc = [&](auto kernel, int smem, int threads, int regs) {
            ok = ok && set_smem(kernel, smem) == cudaSuccess;
            fits = fits && split_fits(kernel, threads, regs);
        };
        auto tc_d = [&](auto d) {
            constexpr int D = decltype(d)::value;
            tc(attn_fwd_tc_kernel<D, 0>, FwdTcLayout<D, 0>::SMEM_BYTES, kFwdTcThreads, FwdTcLayout<D, 0>::REGS_SPLIT);
            tc(attn_fwd_tc_kernel<D, 1>, FwdTcLayout<D, 1>::SMEM_BYTES, kFwdTcThreads, FwdTcLayout<D, 1>::REGS_SPLIT);
            ok = ok && set_smem(attn_few_kernel<D>, FewLayout<D>::SMEM_BYTES) == cudaSuccess;
            tc(attn_dq_tc_kernel<D>, DqLayout<D>::SMEM_BYTES, kBwdTcThreads, kDqRegsSplitTotal);
            tc(attn_dkdv_tc_kernel<D>, DkvLayout<D>::SMEM_BYTES, kBwdTcThreads, kDqRegsSplitTotal);
        };
        tc_d(std::integral_constant<int, 64>());
        tc_d(std::integral_constant<int, 128>());
        auto simt = [&](auto d) {
            constexpr int D = decltype(d)::value;
            ok = ok && set_smem(attn_fwd_simt_kernel<D, 1>, SimtLayout<D>::FWD_BYTES) == cudaSuccess &&
                 set_smem(attn_fwd_simt_kernel<D, 4>, SimtLayout<D>::FWD_BYTES) == cudaSuccess &&
                 set_smem(attn_dkdv_simt_kernel<D>, SimtLayout<D>::DKDV_BYTES) == cudaSuccess &&
                 set_smem(attn_dq_simt_kernel<D>, SimtLayout<D>::DQ_BYTES) == cudaSuccess;
        };
        simt(std::integral_constant<int, 64>());
        simt(std::integral_constant<int, 128>());
        if (!ok) st = LARD_ERR_CUDA;
        else if (!fits) st = LARD_ERR_UNSUPPORTED;  // a build whose register count cannot host the split
    }
    g_dev_status[dev] = st;
    g_ready[dev] = true;
    return st;
}

// ------------------------------------------------------------------ arguments
// One buffer of a call: a strided view, or a flat range (rows of one element).
struct Buffer {
    uintptr_t p = 0;
    long long dim[3] = {1, 1, 1}, stride[3] = {0, 0, 0};  // in bytes, largest stride first
    long long width = 0;                                  // bytes of a row
    bool out = false;
    long long span() const {
        long long s = width;
        for (int k = 0; k < 3; ++k) s += stride[k] * (dim[k] - 1);
        return s;
    }
    bool same_strides(const Buffer& o) const {
        for (int k = 0; k < 3; ++k)
            if (stride[k] != o.stride[k] || dim[k] != o.dim[k]) return false;
        return width == o.width;
    }
};

// Whether some rows of two views of equal strides, whose rows do not overlap
// within one view, overlap: the offset between them is walked down stride by
// stride, where only the nearest multiples can come within a row.
bool rows_meet(long long delta, const Buffer& b, int k) {
    if (k == 3) return delta < b.width && -delta < b.width;
    if (b.dim[k] == 1) return rows_meet(delta, b, k + 1);
    const long long at = -delta / b.stride[k];
    for (long long c = at - 1; c <= at + 1; ++c)
        if (c > -b.dim[k] && c < b.dim[k] && rows_meet(delta + c * b.stride[k], b, k + 1)) return true;
    return false;
}

struct Buffers {
    Buffer b[16];
    int k = 0;
    bool add_view(const lard_attn_view& v, long long B, long long H, long long rows, int d, int elem, bool out,
                  lard_attn_view* clean) {
        if (!v.ptr || !aligned(v.ptr, 16)) return false;
        Buffer x;
        x.p = reinterpret_cast<uintptr_t>(v.ptr);
        x.width = static_cast<long long>(d) * elem;
        x.out = out;
        const long long dims[3] = {B, H, rows}, strides[3] = {v.batch, v.head, v.row};
        long long kept[3];
        for (int a = 0; a < 3; ++a) {
            kept[a] = 0;
            if (dims[a] == 1) continue;  // the stride of a single element is not used
            if (strides[a] < 0 || strides[a] >= (1LL << 40) / elem || strides[a] * elem % 16 != 0) return false;
            kept[a] = strides[a];
        }
        if (rows > 1 && kept[2] < d) return false;
        *clean = lard_attn_view{v.ptr, kept[0], kept[1], kept[2]};
        int order[3] = {0, 1, 2};
        std::sort(order, order + 3, [&](int a, int c) { return kept[a] > kept[c]; });
        double total = static_cast<double>(x.width);
        for (int a = 0; a < 3; ++a) {
            x.dim[a] = dims[order[a]];
            x.stride[a] = kept[order[a]] * elem;
            total += static_cast<double>(x.stride[a]) * static_cast<double>(x.dim[a] - 1);
        }
        if (total > 9.0e18 / 8) return false;  // the address range stays in 60 bits
        if (out) {  // rows of an output may not overlap: each stride passes over what the smaller ones span
            long long span = x.width;
            for (int a = 2; a >= 0; --a) {
                if (x.dim[a] == 1) continue;
                if (x.stride[a] < span) return false;
                span += x.stride[a] * (x.dim[a] - 1);
            }
        }
        b[k++] = x;
        return true;
    }
    void add_flat(const void* p, size_t bytes, bool out) {
        if (!p || bytes == 0) return;
        Buffer x;
        x.p = reinterpret_cast<uintptr_t>(p);
        x.width = static_cast<long long>(bytes);
        x.out = out;
        b[k++] = x;
    }
    bool outputs_disjoint() const {
        for (int i = 0; i < k; ++i)
            for (int j = i + 1; j < k; ++j) {
                if (!b[i].out && !b[j].out) continue;
                if (!overlap(reinterpret_cast<void*>(b[i].p), b[i].span(), reinterpret_cast<void*>(b[j].p), b[j].span()))
                    continue;
                if (!b[i].same_strides(b[j])) return false;
                if (rows_meet(static_cast<long long>(b[j].p) - static_cast<long long>(b[i].p), b[i], 0)) return false;
            }
        return true;
    }
    // Makes the GPU of the first buffer current and sets it up; the others must be on it.
    lard_status select_device() const {
        int dev = -1;
        for (int i = 0; i < k; ++i) {
            cudaPointerAttributes at;
            if (cudaPointerGetAttributes(&at, reinterpret_cast<void*>(b[i].p)) != cudaSuccess) {
                cudaGetLastError();
                return LARD_ERR_CUDA;
            }
            if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) return LARD_ERR_INVALID_ARG;
            if (dev < 0) dev = at.device;
            if (at.device != dev) return LARD_ERR_INVALID_ARG;
        }
        if (cudaSetDevice(dev) != cudaSuccess) return LARD_ERR_CUDA;
        return setup_device(dev);
    }
};

int elem_bytes(lard_dtype t) { return t == LARD_DTYPE_BF16 ? 2 : 4; }

lard_status check_sizes(lard_dtype dtype, int B, int Hq, int Hkv, int n, int d, float tau) {
    if (B < 1 || Hq < 1 || Hkv < 1 || n < 1 || d < 1 || Hq % Hkv != 0) return LARD_ERR_INVALID_ARG;
    if (!(std::isfinite(tau) && tau > 0.f)) return LARD_ERR_INVALID_ARG;
    if (dtype != LARD_DTYPE_BF16 && dtype != LARD_DTYPE_FP32) return LARD_ERR_UNSUPPORTED;
    if (d != 64 && d != 128) return LARD_ERR_UNSUPPORTED;
    if (n > kMaxRows || static_cast<long long>(Hq / Hkv) * n > kMaxRows) return LARD_ERR_INVALID_ARG;
    if (static_cast<long long>(B) * Hq >= (1LL << 30)) return LARD_ERR_INVALID_ARG;
    return LARD_OK;
}

template <typename T>
View<T> view(const lard_attn_view& v) {
    return View<T>{static_cast<T*>(v.ptr), v.batch, v.head, v.row};
}

// Launches a kernel; `after`: it may start beside the kernel before it in the
// call, and itself waits (attn_ptx.cuh) for what it reads of that one's.
template <typename... Params, typename... Args>
lard_status launch(void (*kernel)(Params...), long long grid, int threads, int smem, cudaStream_t stream, bool after,
                   int cluster, Args&&... args) {
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(static_cast<unsigned>(grid));
    c.blockDim = dim3(static_cast<unsigned>(threads));
    c.dynamicSmemBytes = static_cast<size_t>(smem);
    c.stream = stream;
    cudaLaunchAttribute at[2];
    if (cluster > 0) {
        at[c.numAttrs].id = cudaLaunchAttributeClusterDimension;
        at[c.numAttrs].val.clusterDim.x = static_cast<unsigned>(cluster);
        at[c.numAttrs].val.clusterDim.y = at[c.numAttrs].val.clusterDim.z = 1;
        ++c.numAttrs;
    }
    if (after) {
        at[c.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[c.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++c.numAttrs;
    }
    c.attrs = at;
    if (cudaLaunchKernelEx(&c, kernel, std::forward<Args>(args)...) == cudaSuccess) return LARD_OK;
    cudaGetLastError();
    return LARD_ERR_CUDA;
}

// ------------------------------------------------------------------ forward
constexpr long long kSumRowsPerBlock = 8;
// Rows from which a join's warp takes eight (one row: 5.6 us for 4096 rows of eight parts,
// 7.3 for 8192 of four, 10.5 for 16384 of two; eight: 9.9, 7.3 and 7.2 us).
constexpr long long kManyRows = 8192;

long long tiles_of(long long rows, int tile) { return (rows + tile - 1) / tile; }

// One pass over the keys of a call: PB problems per key head of R rows each
// over at most `tiles` key tiles, the key axis dealt to `splits` blocks.
struct Pass {
    enum Kind { kSimt, kSimtFew, kTcRows, kTcKeys, kFew } kind = kSimt;
    long long blocks = 0;  // of one split
    int splits = 0;
    int nseg = 1, seg = 0;  // segments [seg, seg + nseg)
    int shared = 0;         // one problem per key head over all sequences' rows
    int cluster = 1;  // kFew: blocks of a cluster, which share a problem's keys
};

// A forward call: one pass, or two (prefix attention: the shared keys, then
// each sequence's own), and what they leave for the join.
struct FwdPlan {
    Pass pass[2];
    int npass = 0;
    long long rows = 0;  // of the whole call
    int d = 0;
    int partials() const { return pass[0].splits + pass[1].splits; }
    bool join() const { return partials() > 1; }
    size_t part_o() const { return join() ? static_cast<size_t>(partials()) * rows * d * 4 : 0; }
    size_t part_lse() const { return join() ? (static_cast<size_t>(partials()) * rows * 4 + 15) / 16 * 16 : 0; }
    size_t bytes() const { return part_o() + part_lse(); }
    bool grids_fit() const {
        for (int k = 0; k < npass; ++k)
            if (pass[k].blocks * pass[k].splits > INT_MAX) return false;
        return !join() || rows <= INT_MAX;
    }
};

// How many blocks share a long axis of `steps` tiles when there are `blocks`
// without: as many as fill the GPU once, where one set would leave it partly idle.
// Measured, gradients at d = 128 (dQ blocks x dK, dV blocks; us): 64 x 64 (2 heads, 4096 x
// 4096) 122 with one block each, 82 with the two that this gives; 128 x 128 (8 heads, 2048 x
// 2048) 74 with one, 97 to 117 with two on either side.  What it leaves: a long axis where one set
// ends in a short second round.  160 x 640 (10 heads, 2048 x 8192) 394, two or three
// blocks for dQ 366; 80 x 640 (1024 x 8192) 215, three 207 (two 235).
int split_to_fill(long long blocks, long long steps, long long slots) {
    if (blocks >= slots) return 1;
    return static_cast<int>(std::max(1LL, std::min(steps, slots / blocks)));
}

// The same for the CUDA-core kernels, whose blocks are few and long: the number
// with the least time, in us, by a model: rounds of blocks (one an SM: their
// registers, or at 16 rows their shared memory), 4 us and steps of step_us each, and 5 us and the partial sums' way out and back at 5 TB/s where
// there are any.  (dK and dV of 8 heads of 1000 x 2000 rows at d = 128: 530 us with one
// block for each tile, two rounds of 148; 487 us with four.)
int split_simt(long long blocks, long long steps, long long slots, double step_us, double out_bytes) {
    int best = 1;
    double least = 0.0;
    for (long long s = 1; s <= std::min(steps, 64LL); ++s) {
        double cost = tiles_of(blocks * s, static_cast<int>(slots)) * (tiles_of(steps, static_cast<int>(s)) * step_us + 4.0);
        if (s > 1) cost += 5.0 + s * out_bytes * 2.0 / 5.0e6;
        if (s == 1 || cost < least) {
            least = cost;
            best = static_cast<int>(s);
        }
    }
    return best;
}

// CUDA-core pass, in tiles of 64 rows, or of 16 where that is all there are;
// two key tiles a step, 16 us (7 us).
Pass plan_simt(long long problems, long long R, int d, long long tiles) {
    Pass p;
    p.kind = R <= 16 ? Pass::kSimtFew : Pass::kSimt;
    const bool few = p.kind == Pass::kSimtFew;
    p.blocks = problems * tiles_of(R, few ? 16 : lard::attn::kSimtTile);
    p.splits = split_simt(p.blocks, tiles_of(tiles, 2), kSms, few ? 7.0 : 16.0, 4.0 * problems * R * d);
    return p;
}

// Keys of a tile of the tensor-core pass.
int tc_tile(int d) { return d == 64 ? lard::attn::FwdTcLayout<64, 0>::KT : lard::attn::FwdTcLayout<128, 0>::KT; }

// Tensor-core pass.  Up to 128 rows the two streams of a block share them and
// take alternate key tiles; more rows take one tile of rows each.  The number
// of splits is the one that a model of the pass's time gives, in cycles: a
// step (products and exponentials of two tiles) takes 3700 (d = 64: 2 x 64 keys, two blocks
// an SM), or as long as HBM (3400 B a cycle) needs to bring the
// running blocks' tiles where each is read once; a block's beginning and end
// 12000; partial rows are written, read and joined at 3400 B a cycle by a
// kernel of its own, 8000.
// (1 x 4096 rows of 32 heads over 16384 keys, 512 blocks: one split 1.10 ms, two 1.06 ms.)
Pass plan_tc(long long problems, long long R, int d, long long tiles, long long rows) {
    Pass p;
    const bool by_keys = R <= 128;
    p.kind = by_keys ? Pass::kTcKeys : Pass::kTcRows;
    const long long rtiles = tiles_of(R, by_keys ? 128 : 256), slots = d == 64 ? 2 * kSms : kSms;
    p.blocks = problems * rtiles;
    double best = 0.0;
    const long long most = std::max(1LL, std::min(64LL, by_keys ? tiles / 2 : tiles));
    for (long long s = 1; s <= most; ++s) {
        const long long blocks = p.blocks * s, full = blocks / slots, rest = blocks % slots;
        const double steps = static_cast<double>(tiles_of(tiles_of(tiles, s), by_keys ? 2 : 1));
        auto time = [&](long long running) {
            double step = 3700.0;
            if (rtiles == 1) step = std::max(step, (by_keys ? 2 : 1) * 4.0 * tc_tile(d) * d * running / 3400.0);
            return steps * step + 12000.0;
        };
        double cost = full * time(slots) + (rest ? time(rest) : 0.0);
        if (s > 1) cost += 8000.0 + 8.0 * s * rows * d / 3400.0;
        if (s == 1 || cost < best) {
            best = cost;
            p.splits = static_cast<int>(s);
        }
    }
    return p;
}

// Pass of at most 16 rows a problem.  A problem's keys are dealt to a cluster of
// up to eight blocks of four warps, which join their rows without a second
// kernel.  The size is the one with the least time, in us, by a model: three
// blocks an SM run at a time; a warp takes a group of 16 keys in 1 us, or in the
// time that HBM needs for one group of every running warp; a round of blocks
// has 3 us of its own.  (128 problems of 8000 keys at d = 128: 3 blocks each
// fill one round, 84 us; 8 fill 2.3, 97 us.)  Where eight blocks leave
// SMs idle (few problems of many keys), several clusters share a problem and the join
// kernel joins them.
Pass plan_few(long long problems, long long groups, int d) {
    Pass p;
    p.kind = Pass::kFew;
    const long long slots = 3 * kSms;
    double best = 0.0;
    for (int c = 1; c <= 8; ++c) {
        const long long blocks = problems * c, full = blocks / slots, rest = blocks % slots;
        const double rounds = static_cast<double>(tiles_of(groups, lard::attn::kFewWarps * c));
        auto time = [&](long long running) {
            return rounds * std::max(1.0, running * lard::attn::kFewWarps * 64.0 * d / 6.5e6) + 3.0;
        };
        const double cost = full * time(slots) + (rest ? time(rest) : 0.0);
        if (c == 1 || cost < best) {
            best = cost;
            p.cluster = c;
        }
    }
    p.blocks = problems * p.cluster;
    p.splits = 1;
    if (p.blocks < 2 * kSms)
        p.splits = static_cast<int>(std::max(1LL, std::min(slots / p.blocks, groups / (16 * p.cluster * lard::attn::kFewWarps))));
    return p;
}

// The forward work of a call, whatever its type: the views and the key segments.
struct Fwd {
    lard_dtype dtype;
    int B, Hq, Hkv, n, d;
    float tau;
    lard_attn_view q, out, rest;  // rest.ptr may be NULL
    float* lse;
    struct Seg {
        lard_attn_view k, v;
        int rows;
        const int* len;
        int shared, causal;  // shared: one block of keys for all sequences
    } seg[2];
    int nseg;
    long long group_rows() const { return static_cast<long long>(Hq / Hkv) * n; }
};

FwdPlan plan_fwd(const Fwd& f) {
    FwdPlan p;
    p.d = f.d;
    p.rows = static_cast<long long>(f.B) * f.Hkv * f.group_rows();
    const long long own = static_cast<long long>(f.B) * f.Hkv;
    const bool fp32 = f.dtype == LARD_DTYPE_FP32;
    auto add = [&](int seg, int nseg, bool shared) {
        const long long problems = shared ? f.Hkv : own, R = f.group_rows() * (shared ? f.B : 1);
        auto tiles = [&](int tile) {
            long long t = 0;
            for (int s = seg; s < seg + nseg; ++s) t += tiles_of(f.seg[s].rows, tile);
            return t;
        };
        Pass x = fp32                         ? plan_simt(problems, R, f.d, tiles(lard::attn::kSimtTile))
                 : R <= lard::attn::kFewRows ? plan_few(problems, tiles(16), f.d)
                                              : plan_tc(problems, R, f.d, tiles(tc_tile(f.d)), p.rows);
        x.seg = seg;
        x.nseg = nseg;
        x.shared = shared;
        p.pass[p.npass++] = x;
    };
    // A shared prefix is read once for all sequences, in a pass of its own, unless
    // there is one sequence, or so little to read again (from L2) that a pass and a join
    // cost more: they take about 7 us, in which L2 brings some 16 MB to blocks
    // that wait for them.
    const double again = static_cast<double>(f.B) * f.Hkv * f.seg[0].rows * f.d * 2.0 * elem_bytes(f.dtype);
    if (f.nseg == 2 && f.B > 1 && !(f.group_rows() <= lard::attn::kFewRows && again <= 16.0e6)) {
        add(0, 1, true);
        add(1, 1, false);
    } else {
        add(0, f.nseg, f.nseg == 1 && f.B > 1 && f.seg[0].shared);
    }
    return p;
}

// 4-D tensor map of a bf16 tensor with boxes of 64 columns x box_rows rows,
// 128-byte swizzle; rows past the end read as zeros.  A dimension of one
// element, or of one block for all (stride 0), has one entry.
bool make_map(CUtensorMap* m, const lard_attn_view& v, long long B, long long H, long long rows, int d,
              unsigned box_rows = 128) {
    const cuuint64_t line = static_cast<cuuint64_t>(d) * 2;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows),
                          static_cast<cuuint64_t>(v.head ? H : 1), static_cast<cuuint64_t>(v.batch ? B : 1)};
    cuuint64_t strides[3] = {v.row ? static_cast<cuuint64_t>(v.row) * 2 : line,
                             v.head ? static_cast<cuuint64_t>(v.head) * 2 : line,
                             v.batch ? static_cast<cuuint64_t>(v.batch) * 2 : line};
    cuuint32_t box[4] = {64, box_rows, 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.ptr, dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

float log2_factor(float tau) { return static_cast<float>(static_cast<double>(tau) * 1.4426950408889634); }

template <typename T>
FwdArgs<T> fwd_args(const Fwd& f) {
    FwdArgs<T> g;
    g.q = view<const T>(f.q);
    g.out = view<T>(f.out);
    g.rest = view<T>(f.rest);
    g.lse = f.lse;
    for (int s = 0; s < 2; ++s) {
        const Fwd::Seg& x = f.seg[s < f.nseg ? s : 0];
        g.seg[s] = KeySeg<T>{view<const T>(x.k), view<const T>(x.v), x.len, x.rows, x.causal};
    }
    g.nseg = f.nseg;
    g.Hkv = f.Hkv;
    g.G = f.Hq / f.Hkv;
    g.n = f.n;
    g.cfac = log2_factor(f.tau);
    return g;
}

// What the passes' arguments have in common.
template <typename A, typename T>
void pass_args(A& a, const Fwd& f, const FwdPlan& p, const Pass& x, int split0, const FwdArgs<T>& g) {
    a.q = g.q;
    a.out = g.out;
    a.rest = g.rest;
    a.lse = g.lse;
    a.nseg = x.nseg;
    a.PB = x.shared ? 1 : f.B;
    a.Hkv = g.Hkv;
    a.G = g.G;
    a.n = g.n;
    a.R = static_cast<int>(f.group_rows() * (x.shared ? f.B : 1));
    a.splits = x.splits;
    a.split0 = split0;
    a.second = split0 > 0;
    a.join = p.join();
    a.rows = p.rows;
    a.part_o = g.part_o;
    a.part_lse = g.part_lse;
    a.cfac = g.cfac;
}

template <int D>
lard_status run_simt(const Fwd& f, const FwdPlan& p, const Pass& x, int split0, const FwdArgs<float>& g,
                     cudaStream_t stream) {
    using namespace lard::attn;
    FwdArgs<float> a;
    pass_args(a, f, p, x, split0, g);
    a.seg[0] = g.seg[x.seg];
    a.seg[1] = g.seg[x.nseg > 1 ? x.seg + 1 : x.seg];
    return launch(x.kind == Pass::kSimtFew ? attn_fwd_simt_kernel<D, 1> : attn_fwd_simt_kernel<D, 4>, x.blocks * x.splits,
                  kSimtThreads, SimtLayout<D>::FWD_BYTES, stream, a.second, 0, a);
}

// The key segments of a pass for TMA loads of box_rows rows.
bool make_segs(lard::attn::TcSeg (&seg)[2], const Fwd& f, const Pass& x, unsigned box_rows) {
    for (int k = 0; k < x.nseg; ++k) {
        const Fwd::Seg& y = f.seg[x.seg + k];
        lard::attn::TcSeg& s = seg[k];
        if (!make_map(&s.k, y.k, y.shared ? 1 : f.B, f.Hkv, y.rows, f.d, box_rows) ||
            !make_map(&s.v, y.v, y.shared ? 1 : f.B, f.Hkv, y.rows, f.d, box_rows))
            return false;
        s.len = y.len;
        s.cap = y.rows;
        s.causal = y.causal;
        s.khead = y.k.head != 0;
        s.kbatch = y.k.batch != 0;
        s.vhead = y.v.head != 0;
        s.vbatch = y.v.batch != 0;
    }
    if (x.nseg == 1) seg[1] = seg[0];
    return true;
}

template <int D>
lard_status run_few(const Fwd& f, const FwdPlan& p, const Pass& x, int split0, const FwdArgs<bf16>& g,
                    cudaStream_t stream) {
    using namespace lard::attn;
    FewArgs a;
    pass_args(a, f, p, x, split0, g);
    if (!make_segs(a.seg, f, x, 16)) return LARD_ERR_INVALID_ARG;
    a.cluster = x.cluster;
    a.wait_ns = kWaitLimitNs;
    a.drain_ns = kDrainLimitNs;
    return launch(attn_few_kernel<D>, x.blocks * x.splits, 32 * kFewWarps, FewLayout<D>::SMEM_BYTES, stream, a.second,
                  x.cluster, a);
}

template <int D>
lard_status run_tc(const Fwd& f, const FwdPlan& p, const Pass& x, int split0, const FwdArgs<bf16>& g,
                   cudaStream_t stream) {
    using namespace lard::attn;
    TcFwdArgs a;
    pass_args(a, f, p, x, split0, g);
    if (!make_segs(a.seg, f, x, FwdTcLayout<D, 0>::KT)) return LARD_ERR_INVALID_ARG;
    a.wait_ns = kWaitLimitNs;
    a.drain_ns = kDrainLimitNs;
    return x.kind == Pass::kTcKeys ? launch(attn_fwd_tc_kernel<D, 1>, x.blocks * x.splits, kFwdTcThreads,
                                            FwdTcLayout<D, 1>::SMEM_BYTES, stream, a.second, 0, a)
                                   : launch(attn_fwd_tc_kernel<D, 0>, x.blocks * x.splits, kFwdTcThreads,
                                            FwdTcLayout<D, 0>::SMEM_BYTES, stream, a.second, 0, a);
}

template <typename T, int D>
lard_status run_fwd(const Fwd& f, const FwdPlan& p, void* ws, cudaStream_t stream) {
    using namespace lard::attn;
    FwdArgs<T> g = fwd_args<T>(f);
    g.splits = p.partials();
    g.rows = p.rows;
    g.part_o = static_cast<float*>(ws);
    g.part_lse = reinterpret_cast<float*>(static_cast<char*>(ws) + p.part_o());
    int split0 = 0;
    for (int k = 0; k < p.npass; ++k) {
        const Pass& x = p.pass[k];
        lard_status st = LARD_OK;
        if constexpr (std::is_same<T, float>::value) st = run_simt<D>(f, p, x, split0, g, stream);
        else if (x.kind == Pass::kFew) st = run_few<D>(f, p, x, split0, g, stream);
        else st = run_tc<D>(f, p, x, split0, g, stream);
        if (st != LARD_OK) return st;
        split0 += x.splits;
    }
    if (!p.join()) return LARD_OK;
    return p.rows >= kManyRows ? launch(attn_join_kernel<T, D, 8>, tiles_of(p.rows, 64), kJoinThreads, 0, stream, true, 0, g)
                               : launch(attn_join_kernel<T, D, 1>, tiles_of(p.rows, 8), kJoinThreads, 0, stream, true, 0, g);
}

Fwd cross_work(const lard_cross_attn& a, const lard_attn_view* v = nullptr) {
    Fwd f{};
    f.dtype = a.dtype;
    f.B = a.B;
    f.Hq = a.Hq;
    f.Hkv = a.Hkv;
    f.n = a.n;
    f.d = a.d;
    f.tau = a.tau;
    f.lse = a.lse;
    f.nseg = 1;
    f.seg[0].rows = a.m;
    f.seg[0].len = a.k_len;
    if (v) {
        f.q = v[0];
        f.seg[0].k = v[1];
        f.seg[0].v = v[2];
        f.out = v[3];
        f.rest = v[4];
    }
    return f;
}

Fwd prefix_work(const lard_prefix_attn_args& a, const lard_attn_view* v = nullptr) {
    Fwd f{};
    f.dtype = a.dtype;
    f.B = a.B;
    f.Hq = a.Hq;
    f.Hkv = a.Hkv;
    f.n = a.n;
    f.d = a.d;
    f.tau = a.tau;
    f.lse = a.lse;
    if (v) {
        f.q = v[0];
        f.out = v[5];
    }
    for (int own = 0; own < 2; ++own) {
        const int rows = own ? a.S : a.P;
        if (rows == 0) continue;
        Fwd::Seg& s = f.seg[f.nseg++];
        s.rows = rows;
        s.len = own ? a.s_len : nullptr;
        s.shared = !own;
        s.causal = own;
        if (v) {
            s.k = v[1 + 2 * own];
            s.v = v[2 + 2 * own];
        }
    }
    return f;
}

lard_status cross_sizes(const lard_cross_attn* a) {
    if (!a) return LARD_ERR_INVALID_ARG;
    lard_status st = check_sizes(a->dtype, a->B, a->Hq, a->Hkv, a->n, a->d, a->tau);
    if (st != LARD_OK) return st;
    if (a->m < 1 || a->m > kMaxRows) return LARD_ERR_INVALID_ARG;
    return plan_fwd(cross_work(*a)).grids_fit() ? LARD_OK : LARD_ERR_INVALID_ARG;
}

lard_status prefix_sizes(const lard_prefix_attn_args* a) {
    if (!a) return LARD_ERR_INVALID_ARG;
    lard_status st = check_sizes(a->dtype, a->B, a->Hq, a->Hkv, a->n, a->d, a->tau);
    if (st != LARD_OK) return st;
    if (a->P < 0 || a->S < 0 || (a->P == 0 && a->S == 0) || a->P > kMaxRows || a->S > kMaxRows)
        return LARD_ERR_INVALID_ARG;
    if (static_cast<long long>(a->B) * (a->Hq / a->Hkv) * a->n > kMaxRows) return LARD_ERR_INVALID_ARG;
    return plan_fwd(prefix_work(*a)).grids_fit() ? LARD_OK : LARD_ERR_INVALID_ARG;
}

bool workspace_ok(const void* ws, size_t have, size_t need) {
    return need == 0 || (ws && aligned(ws, 16) && have >= need);
}

lard_status launch_fwd(const Fwd& f, const FwdPlan& p, void* ws, cudaStream_t stream) {
    if (f.dtype == LARD_DTYPE_BF16)
        return f.d == 64 ? run_fwd<bf16, 64>(f, p, ws, stream) : run_fwd<bf16, 128>(f, p, ws, stream);
    return f.d == 64 ? run_fwd<float, 64>(f, p, ws, stream) : run_fwd<float, 128>(f, p, ws, stream);
}

// ------------------------------------------------------------------ backward
// Layout of a backward call: splits of the key axis for dQ and of the row axis
// for dK and dV, and the workspace: delta, then the partial sums.
struct BwdPlan {
    long long qblocks = 0, kblocks = 0;  // of one split
    int qsplits = 1, ksplits = 1;
    size_t delta = 0, part_q = 0, part_kv = 0;  // bytes; part_kv of dK and of dV each
    long long sum_rows = 0;
    size_t bytes() const { return delta + part_q + 2 * part_kv; }
    bool grids_fit() const {
        return qblocks * qsplits <= INT_MAX && kblocks * ksplits <= INT_MAX && tiles_of(sum_rows, kSumRowsPerBlock) <= INT_MAX;
    }
};

BwdPlan plan_bwd(const lard_cross_attn& a) {
    BwdPlan p;
    const long long BH = static_cast<long long>(a.B) * a.Hkv, R = static_cast<long long>(a.Hq / a.Hkv) * a.n;
    p.delta = (static_cast<size_t>(BH) * R * 4 + 15) / 16 * 16;
    const int tile = a.dtype == LARD_DTYPE_FP32 ? lard::attn::kSimtTile : 128;
    p.qblocks = BH * tiles_of(R, tile);
    p.kblocks = BH * tiles_of(a.m, tile);
    const long long qsteps = tiles_of(a.m, tile), ksteps = tiles_of(R, tile);
    if (a.dtype == LARD_DTYPE_FP32) {
        p.qsplits = split_simt(p.qblocks, qsteps, kSms, 12.0, 4.0 * BH * R * a.d);
        p.ksplits = split_simt(p.kblocks, ksteps, kSms, 16.0, 8.0 * BH * a.m * a.d);
    } else {
        p.qsplits = split_to_fill(p.qblocks, qsteps, kSms);
        p.ksplits = split_to_fill(p.kblocks, ksteps, kSms);
    }
    if (p.qsplits > 1) {
        p.part_q = static_cast<size_t>(p.qsplits) * BH * R * a.d * 4;
        p.sum_rows += BH * R;
    }
    if (p.ksplits > 1) {
        p.part_kv = static_cast<size_t>(p.ksplits) * BH * a.m * a.d * 4;
        p.sum_rows += 2 * BH * a.m;
    }
    return p;
}

// delta and the partial sums' places in the workspace.
template <typename Args>
void take_bwd_workspace(Args& g, const BwdPlan& p, void* ws) {
    char* w = static_cast<char*>(ws);
    g.delta = reinterpret_cast<float*>(w);
    g.part_q = reinterpret_cast<float*>(w + p.delta);
    g.part_k = reinterpret_cast<float*>(w + p.delta + p.part_q);
    g.part_v = reinterpret_cast<float*>(w + p.delta + p.part_q + p.part_kv);
    g.qsplits = p.qsplits;
    g.ksplits = p.ksplits;
}

// Adds the partial sums that a backward call left.
template <typename T, int D>
lard_status run_sums(const lard_cross_attn& a, const BwdPlan& p, const lard_attn_view (&v)[9], const float* part_q,
              const float* part_k, const float* part_v, cudaStream_t stream) {
    using namespace lard::attn;
    if (p.sum_rows == 0) return LARD_OK;
    SumArgs<T> s;
    s.jobs = 0;
    if (p.qsplits > 1)
        s.job[s.jobs++] = {part_q, view<T>(v[5]), p.qsplits, a.Hq, a.n, static_cast<long long>(a.B) * a.Hq * a.n, a.tau};
    if (p.ksplits > 1) {
        s.job[s.jobs++] = {part_k, view<T>(v[6]), p.ksplits, a.Hkv, a.m, static_cast<long long>(a.B) * a.Hkv * a.m, a.tau};
        s.job[s.jobs++] = {part_v, view<T>(v[7]), p.ksplits, a.Hkv, a.m, static_cast<long long>(a.B) * a.Hkv * a.m, 1.f};
    }
    return launch(attn_sum_kernel<T, D>, tiles_of(p.sum_rows, kSumRowsPerBlock), 256, 0, stream, true, 0, s);
}

template <int D>
lard_status run_bwd_tc(const lard_cross_attn& a, const BwdPlan& p, const lard_attn_view (&v)[9], void* ws,
                       cudaStream_t stream) {
    using namespace lard::attn;
    TcBwdArgs g;
    if (!make_map(&g.k, v[1], a.B, a.Hkv, a.m, D) || !make_map(&g.v, v[2], a.B, a.Hkv, a.m, D) ||
        !make_map(&g.q64, v[0], a.B, a.Hq, a.n, D, kUnit) || !make_map(&g.do64, v[4], a.B, a.Hq, a.n, D, kUnit))
        return LARD_ERR_INVALID_ARG;
    g.q = view<const bf16>(v[0]);
    g.out = view<const bf16>(v[3]);
    g.rest = view<const bf16>(v[8]);
    g.dout = view<const bf16>(v[4]);
    g.dq = view<bf16>(v[5]);
    g.dk = view<bf16>(v[6]);
    g.dv = view<bf16>(v[7]);
    g.lse = a.lse;
    take_bwd_workspace(g, p, ws);
    g.len = a.k_len;
    g.m = a.m;
    g.B = a.B;
    g.Hkv = a.Hkv;
    g.G = a.Hq / a.Hkv;
    g.n = a.n;
    g.khead = v[1].head != 0;
    g.kbatch = v[1].batch != 0;
    g.vhead = v[2].head != 0;
    g.vbatch = v[2].batch != 0;
    g.qhead = v[0].head != 0;
    g.qbatch = v[0].batch != 0;
    g.dohead = v[4].head != 0;
    g.dobatch = v[4].batch != 0;
    g.cfac = log2_factor(a.tau);
    g.tau = a.tau;
    g.wait_ns = kWaitLimitNs;
    g.drain_ns = kDrainLimitNs;
    lard_status st =
        launch(attn_dq_tc_kernel<D>, p.qblocks * p.qsplits, kBwdTcThreads, DqLayout<D>::SMEM_BYTES, stream, false, 0, g);
    if (st == LARD_OK)
        st = launch(attn_dkdv_tc_kernel<D>, p.kblocks * p.ksplits, kBwdTcThreads, DkvLayout<D>::SMEM_BYTES, stream, true, 0, g);
    return st == LARD_OK ? run_sums<bf16, D>(a, p, v, g.part_q, g.part_k, g.part_v, stream) : st;
}

template <int D>
lard_status run_bwd_simt(const lard_cross_attn& a, const BwdPlan& p, const lard_attn_view (&v)[9], void* ws,
                         cudaStream_t stream) {
    using namespace lard::attn;
    SimtBwdArgs g;
    g.q = view<const float>(v[0]);
    g.k = view<const float>(v[1]);
    g.v = view<const float>(v[2]);
    g.out = view<const float>(v[3]);
    g.dout = view<const float>(v[4]);
    g.dq = view<float>(v[5]);
    g.dk = view<float>(v[6]);
    g.dv = view<float>(v[7]);
    g.lse = a.lse;
    take_bwd_workspace(g, p, ws);
    g.len = a.k_len;
    g.m = a.m;
    g.B = a.B;
    g.Hkv = a.Hkv;
    g.G = a.Hq / a.Hkv;
    g.n = a.n;
    g.cfac = log2_factor(a.tau);
    g.tau = a.tau;
    lard_status st =
        launch(attn_dq_simt_kernel<D>, p.qblocks * p.qsplits, kSimtThreads, SimtLayout<D>::DQ_BYTES, stream, false, 0, g);
    if (st == LARD_OK)
        st = launch(attn_dkdv_simt_kernel<D>, p.kblocks * p.ksplits, kSimtThreads, SimtLayout<D>::DKDV_BYTES, stream, true, 0, g);
    return st == LARD_OK ? run_sums<float, D>(a, p, v, g.part_q, g.part_k, g.part_v, stream) : st;
}

lard_status launch_bwd(const lard_cross_attn& a, const BwdPlan& p, const lard_attn_view (&v)[9], void* ws,
                       cudaStream_t stream) {
    if (a.dtype == LARD_DTYPE_BF16)
        return a.d == 64 ? run_bwd_tc<64>(a, p, v, ws, stream) : run_bwd_tc<128>(a, p, v, ws, stream);
    return a.d == 64 ? run_bwd_simt<64>(a, p, v, ws, stream) : run_bwd_simt<128>(a, p, v, ws, stream);
}

}  // namespace

extern "C" {

size_t lard_cross_attn_fwd_workspace_bytes(const lard_cross_attn* a) {
    return cross_sizes(a) == LARD_OK ? plan_fwd(cross_work(*a)).bytes() : 0;
}

size_t lard_cross_attn_bwd_workspace_bytes(const lard_cross_attn* a) {
    return cross_sizes(a) == LARD_OK && plan_bwd(*a).grids_fit() ? plan_bwd(*a).bytes() : 0;
}

size_t lard_prefix_attn_workspace_bytes(const lard_prefix_attn_args* a) {
    return prefix_sizes(a) == LARD_OK ? plan_fwd(prefix_work(*a)).bytes() : 0;
}

lard_status lard_cross_attn_fwd(const lard_cross_attn* a, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
    NvtxRange range("lard cross attention");
    lard_status st = cross_sizes(a);
    if (st != LARD_OK) return st;
    const int e = elem_bytes(a->dtype);
    Buffers bufs;
    lard_attn_view v[5] = {};
    const bool rest = a->dtype == LARD_DTYPE_BF16 && a->rest.ptr;
    if (!bufs.add_view(a->q, a->B, a->Hq, a->n, a->d, e, false, &v[0]) ||
        !bufs.add_view(a->k, a->B, a->Hkv, a->m, a->d, e, false, &v[1]) ||
        !bufs.add_view(a->v, a->B, a->Hkv, a->m, a->d, e, false, &v[2]) ||
        !bufs.add_view(a->out, a->B, a->Hq, a->n, a->d, e, true, &v[3]) ||
        (rest && !bufs.add_view(a->rest, a->B, a->Hq, a->n, a->d, e, true, &v[4])))
        return LARD_ERR_INVALID_ARG;
    if (!a->lse || !aligned(a->lse, 4) || (a->k_len && !aligned(a->k_len, 4))) return LARD_ERR_INVALID_ARG;
    const Fwd work = cross_work(*a, v);
    const FwdPlan plan = plan_fwd(work);
    const size_t need = plan.bytes();
    if (!workspace_ok(workspace, workspace_bytes, need)) return LARD_ERR_INVALID_ARG;
    bufs.add_flat(a->lse, static_cast<size_t>(a->B) * a->Hq * a->n * 4, true);
    bufs.add_flat(a->k_len, static_cast<size_t>(a->B) * 4, false);
    bufs.add_flat(workspace, need, true);
    if (!bufs.outputs_disjoint()) return LARD_ERR_INVALID_ARG;
    DeviceGuard guard;
    st = bufs.select_device();
    if (st != LARD_OK) return st;
    return launch_fwd(work, plan, workspace, stream);
}

lard_status lard_cross_attn_bwd(const lard_cross_attn* a, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
    NvtxRange range("lard cross attention, gradients");
    lard_status st = cross_sizes(a);
    if (st != LARD_OK) return st;
    const int e = elem_bytes(a->dtype);
    Buffers bufs;
    lard_attn_view v[9] = {};
    const bool rest = a->dtype == LARD_DTYPE_BF16 && a->rest.ptr;
    if (!bufs.add_view(a->q, a->B, a->Hq, a->n, a->d, e, false, &v[0]) ||
        !bufs.add_view(a->k, a->B, a->Hkv, a->m, a->d, e, false, &v[1]) ||
        !bufs.add_view(a->v, a->B, a->Hkv, a->m, a->d, e, false, &v[2]) ||
        !bufs.add_view(a->out, a->B, a->Hq, a->n, a->d, e, false, &v[3]) ||
        !bufs.add_view(a->dout, a->B, a->Hq, a->n, a->d, e, false, &v[4]) ||
        !bufs.add_view(a->dq, a->B, a->Hq, a->n, a->d, e, true, &v[5]) ||
        !bufs.add_view(a->dk, a->B, a->Hkv, a->m, a->d, e, true, &v[6]) ||
        !bufs.add_view(a->dv, a->B, a->Hkv, a->m, a->d, e, true, &v[7]) ||
        (rest && !bufs.add_view(a->rest, a->B, a->Hq, a->n, a->d, e, false, &v[8])))
        return LARD_ERR_INVALID_ARG;
    if (!a->lse || !aligned(a->lse, 4) || (a->k_len && !aligned(a->k_len, 4))) return LARD_ERR_INVALID_ARG;
    const BwdPlan plan = plan_bwd(*a);
    if (!plan.grids_fit()) return LARD_ERR_INVALID_ARG;
    const size_t need = plan.bytes();
    if (!workspace_ok(workspace, workspace_bytes, need)) return LARD_ERR_INVALID_ARG;
    bufs.add_flat(a->lse, static_cast<size_t>(a->B) * a->Hq * a->n * 4, false);
    bufs.add_flat(a->k_len, static_cast<size_t>(a->B) * 4, false);
    bufs.add_flat(workspace, need, true);
    if (!bufs.outputs_disjoint()) return LARD_ERR_INVALID_ARG;
    DeviceGuard guard;
    st = bufs.select_device();
    if (st != LARD_OK) return st;
    return launch_bwd(*a, plan, v, workspace, stream);
}

lard_status lard_prefix_attn(const lard_prefix_attn_args* a, void* workspace, size_t workspace_bytes,
                             cudaStream_t stream) {
    NvtxRange range("lard prefix attention");
    lard_status st = prefix_sizes(a);
    if (st != LARD_OK) return st;
    const int e = elem_bytes(a->dtype);
    Buffers bufs;
    lard_attn_view v[6] = {};
    if (!bufs.add_view(a->q, a->B, a->Hq, a->n, a->d, e, false, &v[0])) return LARD_ERR_INVALID_ARG;
    if (a->P > 0 && (!bufs.add_view(a->kp, 1, a->Hkv, a->P, a->d, e, false, &v[1]) ||
                     !bufs.add_view(a->vp, 1, a->Hkv, a->P, a->d, e, false, &v[2])))
        return LARD_ERR_INVALID_ARG;
    if (a->S > 0 && (!bufs.add_view(a->ks, a->B, a->Hkv, a->S, a->d, e, false, &v[3]) ||
                     !bufs.add_view(a->vs, a->B, a->Hkv, a->S, a->d, e, false, &v[4])))
        return LARD_ERR_INVALID_ARG;
    if (!bufs.add_view(a->out, a->B, a->Hq, a->n, a->d, e, true, &v[5])) return LARD_ERR_INVALID_ARG;
    if (!a->lse || !aligned(a->lse, 4) || (a->S > 0 && a->s_len && !aligned(a->s_len, 4))) return LARD_ERR_INVALID_ARG;
    const Fwd work = prefix_work(*a, v);
    const FwdPlan plan = plan_fwd(work);
    const size_t need = plan.bytes();
    if (!workspace_ok(workspace, workspace_bytes, need)) return LARD_ERR_INVALID_ARG;
    bufs.add_flat(a->lse, static_cast<size_t>(a->B) * a->Hq * a->n * 4, true);
    if (a->S > 0) bufs.add_flat(a->s_len, static_cast<size_t>(a->B) * 4, false);
    bufs.add_flat(workspace, need, true);
    if (!bufs.outputs_disjoint()) return LARD_ERR_INVALID_ARG;
    DeviceGuard guard;
    st = bufs.select_device();
    if (st != LARD_OK) return st;
    return launch_fwd(work, plan, workspace, stream);
}

lard_status lard_attn_device_status(cudaStream_t stream, unsigned int* fault_bits) {
    if (cudaStreamSynchronize(stream) != cudaSuccess) return LARD_ERR_CUDA;
    // The fault word of the stream's GPU, which need not be the current device.
    int dev = 0;
    if (cudaStreamGetDevice(stream, &dev) != cudaSuccess) return LARD_ERR_CUDA;
    DeviceGuard guard;
    if (cudaSetDevice(dev) != cudaSuccess) return LARD_ERR_CUDA;
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, lard::g_lard_fault, sizeof(v)) != cudaSuccess) return LARD_ERR_CUDA;
    if (fault_bits) *fault_bits = v;
    if (v) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(lard::g_lard_fault, &zero, sizeof(zero)) != cudaSuccess) return LARD_ERR_CUDA;
        return LARD_ERR_TIMEOUT;
    }
    return LARD_OK;
}

}  // extern "C"
