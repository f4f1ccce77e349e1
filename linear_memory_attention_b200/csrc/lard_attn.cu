// lard_attn.cu -- the C ABI of liblard_attn (declared in include/lard_attn.h):
// argument checks, per-device setup and kernel launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "lard_attn.h"
#include "lard_host.h"
#include "lard_kernel_common.cuh"
#include "attn/attn_common.cuh"
#include "attn/attn_simt.cuh"

namespace {

using lard::attn::BwdArgs;
using lard::attn::FwdArgs;
using lard::attn::KeySeg;
using lard::attn::View;
using bf16 = __nv_bfloat16;

constexpr int kMaxDevices = 64;
constexpr int kSms = 148;  // of a B200: plans depend on sizes alone, so that a workspace can be sized without a GPU
constexpr int kMaxRows = INT_MAX - 255;

std::mutex g_mu;
bool g_ready[kMaxDevices];
lard_status g_dev_status[kMaxDevices];

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
    if (st == LARD_OK) {
        using namespace lard::attn;
        bool ok = true;
        auto simt = [&](auto t, auto d) {
            using T = decltype(t);
            constexpr int D = decltype(d)::value;
            ok = ok && set_smem(attn_fwd_simt_kernel<T, D>, SimtLayout<D>::FWD_BYTES) == cudaSuccess &&
                 set_smem(attn_dkdv_simt_kernel<T, D>, SimtLayout<D>::BWD_BYTES) == cudaSuccess &&
                 set_smem(attn_dq_simt_kernel<T, D>, SimtLayout<D>::BWD_BYTES) == cudaSuccess;
        };
        simt(float(), std::integral_constant<int, 64>());
        simt(float(), std::integral_constant<int, 128>());
        simt(bf16(), std::integral_constant<int, 64>());
        simt(bf16(), std::integral_constant<int, 128>());
        if (!ok) st = LARD_ERR_CUDA;
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

// ------------------------------------------------------------------ forward
// How a forward pass over `keys` keys at most (two segments' tiles) is laid out.
struct FwdPlan {
    long long rtiles, blocks, rows;
    int splits;
    size_t part_o, part_lse;  // bytes
    size_t bytes() const { return part_o + part_lse; }
};

FwdPlan plan_fwd(long long BH, long long R, int d, long long key_tiles) {
    FwdPlan p;
    p.rows = BH * R;
    p.rtiles = (R + lard::attn::kSimtTile - 1) / lard::attn::kSimtTile;
    p.blocks = BH * p.rtiles;
    // Fewer blocks than SMs: the key tiles of each are dealt to several blocks, two an SM in all.
    long long splits = 1;
    if (p.blocks < kSms) splits = std::max(1LL, std::min(key_tiles, 2 * kSms / p.blocks));
    p.splits = static_cast<int>(splits);
    p.part_o = splits > 1 ? static_cast<size_t>(splits) * p.rows * d * 4 : 0;
    p.part_lse = splits > 1 ? (static_cast<size_t>(splits) * p.rows * 4 + 15) / 16 * 16 : 0;
    return p;
}

template <typename T, int D>
void launch_fwd(FwdArgs<T>& g, const FwdPlan& p, void* ws, cudaStream_t s) {
    using namespace lard::attn;
    g.splits = p.splits;
    g.part_o = static_cast<float*>(ws);
    g.part_lse = reinterpret_cast<float*>(static_cast<char*>(ws) + p.part_o);
    attn_fwd_simt_kernel<T, D><<<static_cast<unsigned>(p.blocks * p.splits), kSimtThreads, SimtLayout<D>::FWD_BYTES, s>>>(g);
    if (p.splits > 1) attn_join_kernel<T, D><<<static_cast<unsigned>((p.rows + 7) / 8), 256, 0, s>>>(g);
}

long long key_tiles(int rows) { return (static_cast<long long>(rows) + lard::attn::kSimtTile - 1) / lard::attn::kSimtTile; }

FwdPlan cross_plan(const lard_cross_attn& a) {
    return plan_fwd(static_cast<long long>(a.B) * a.Hkv, static_cast<long long>(a.Hq / a.Hkv) * a.n, a.d, key_tiles(a.m));
}

FwdPlan prefix_plan(const lard_prefix_attn_args& a) {
    return plan_fwd(static_cast<long long>(a.B) * a.Hkv, static_cast<long long>(a.Hq / a.Hkv) * a.n, a.d,
                    key_tiles(a.P) + key_tiles(a.S));
}

lard_status cross_sizes(const lard_cross_attn* a) {
    if (!a) return LARD_ERR_INVALID_ARG;
    lard_status st = check_sizes(a->dtype, a->B, a->Hq, a->Hkv, a->n, a->d, a->tau);
    if (st != LARD_OK) return st;
    if (a->m < 1 || a->m > kMaxRows) return LARD_ERR_INVALID_ARG;
    const FwdPlan p = cross_plan(*a);
    if (p.blocks * p.splits > INT_MAX || (p.rows + 7) / 8 > INT_MAX ||
        static_cast<long long>(a->B) * a->Hkv * key_tiles(a->m) > INT_MAX)
        return LARD_ERR_INVALID_ARG;
    return LARD_OK;
}

lard_status prefix_sizes(const lard_prefix_attn_args* a) {
    if (!a) return LARD_ERR_INVALID_ARG;
    lard_status st = check_sizes(a->dtype, a->B, a->Hq, a->Hkv, a->n, a->d, a->tau);
    if (st != LARD_OK) return st;
    if (a->P < 0 || a->S < 0 || (a->P == 0 && a->S == 0) || a->P > kMaxRows || a->S > kMaxRows)
        return LARD_ERR_INVALID_ARG;
    const FwdPlan p = prefix_plan(*a);
    if (p.blocks * p.splits > INT_MAX || (p.rows + 7) / 8 > INT_MAX) return LARD_ERR_INVALID_ARG;
    return LARD_OK;
}

bool workspace_ok(const void* ws, size_t have, size_t need) {
    return need == 0 || (ws && aligned(ws, 16) && have >= need);
}

template <typename T, int D>
void cross_fwd(const lard_cross_attn& a, const lard_attn_view (&v)[4], void* ws, cudaStream_t stream) {
    FwdArgs<T> g;
    g.q = View<const T>{static_cast<const T*>(v[0].ptr), v[0].batch, v[0].head, v[0].row};
    g.out = view<T>(v[3]);
    g.lse = a.lse;
    g.seg[0] = KeySeg<T>{view<const T>(v[1]), view<const T>(v[2]), a.k_len, a.m, 0};
    g.seg[1] = g.seg[0];
    g.nseg = 1;
    g.B = a.B;
    g.Hkv = a.Hkv;
    g.G = a.Hq / a.Hkv;
    g.n = a.n;
    g.cfac = static_cast<float>(static_cast<double>(a.tau) * 1.4426950408889634);
    launch_fwd<T, D>(g, cross_plan(a), ws, stream);
}

template <typename T, int D>
void prefix_fwd(const lard_prefix_attn_args& a, const lard_attn_view (&v)[6], void* ws, cudaStream_t stream) {
    FwdArgs<T> g;
    g.q = view<const T>(v[0]);
    g.out = view<T>(v[5]);
    g.lse = a.lse;
    g.nseg = 0;
    if (a.P > 0) g.seg[g.nseg++] = KeySeg<T>{view<const T>(v[1]), view<const T>(v[2]), nullptr, a.P, 0};
    if (a.S > 0) g.seg[g.nseg++] = KeySeg<T>{view<const T>(v[3]), view<const T>(v[4]), a.s_len, a.S, 1};
    if (g.nseg == 1) g.seg[1] = g.seg[0];
    g.B = a.B;
    g.Hkv = a.Hkv;
    g.G = a.Hq / a.Hkv;
    g.n = a.n;
    g.cfac = static_cast<float>(static_cast<double>(a.tau) * 1.4426950408889634);
    launch_fwd<T, D>(g, prefix_plan(a), ws, stream);
}

// ------------------------------------------------------------------ backward
size_t bwd_bytes(const lard_cross_attn& a) {
    return (static_cast<size_t>(a.B) * a.Hq * a.n * 4 + 15) / 16 * 16;  // delta
}

template <typename T, int D>
void cross_bwd(const lard_cross_attn& a, const lard_attn_view (&v)[8], void* ws, cudaStream_t stream) {
    using namespace lard::attn;
    BwdArgs<T> g;
    g.q = view<const T>(v[0]);
    g.k = view<const T>(v[1]);
    g.v = view<const T>(v[2]);
    g.out = view<const T>(v[3]);
    g.dout = view<const T>(v[4]);
    g.dq = view<T>(v[5]);
    g.dk = view<T>(v[6]);
    g.dv = view<T>(v[7]);
    g.lse = a.lse;
    g.delta = static_cast<float*>(ws);
    g.len = a.k_len;
    g.m = a.m;
    g.B = a.B;
    g.Hkv = a.Hkv;
    g.G = a.Hq / a.Hkv;
    g.n = a.n;
    g.cfac = static_cast<float>(static_cast<double>(a.tau) * 1.4426950408889634);
    g.tau = a.tau;
    const long long BH = static_cast<long long>(a.B) * a.Hkv, R = static_cast<long long>(g.G) * a.n;
    const long long rtiles = (R + kSimtTile - 1) / kSimtTile;
    attn_delta_kernel<T, D><<<static_cast<unsigned>((BH * R + 7) / 8), 256, 0, stream>>>(g);
    attn_dkdv_simt_kernel<T, D><<<static_cast<unsigned>(BH * key_tiles(a.m)), kSimtThreads, SimtLayout<D>::BWD_BYTES, stream>>>(g);
    attn_dq_simt_kernel<T, D><<<static_cast<unsigned>(BH * rtiles), kSimtThreads, SimtLayout<D>::BWD_BYTES, stream>>>(g);
}

#define LARD_ATTN_DISPATCH(dtype, d, F, ...)                         \
    do {                                                             \
        if ((dtype) == LARD_DTYPE_BF16) {                            \
            if ((d) == 64) F<bf16, 64>(__VA_ARGS__);                 \
            else F<bf16, 128>(__VA_ARGS__);                          \
        } else {                                                     \
            if ((d) == 64) F<float, 64>(__VA_ARGS__);                \
            else F<float, 128>(__VA_ARGS__);                         \
        }                                                            \
    } while (0)

}  // namespace

extern "C" {

size_t lard_cross_attn_fwd_workspace_bytes(const lard_cross_attn* a) {
    return cross_sizes(a) == LARD_OK ? cross_plan(*a).bytes() : 0;
}

size_t lard_cross_attn_bwd_workspace_bytes(const lard_cross_attn* a) {
    return cross_sizes(a) == LARD_OK ? bwd_bytes(*a) : 0;
}

size_t lard_prefix_attn_workspace_bytes(const lard_prefix_attn_args* a) {
    return prefix_sizes(a) == LARD_OK ? prefix_plan(*a).bytes() : 0;
}

lard_status lard_cross_attn_fwd(const lard_cross_attn* a, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
    NvtxRange range("lard cross attention");
    lard_status st = cross_sizes(a);
    if (st != LARD_OK) return st;
    const int e = elem_bytes(a->dtype);
    Buffers bufs;
    lard_attn_view v[4];
    if (!bufs.add_view(a->q, a->B, a->Hq, a->n, a->d, e, false, &v[0]) ||
        !bufs.add_view(a->k, a->B, a->Hkv, a->m, a->d, e, false, &v[1]) ||
        !bufs.add_view(a->v, a->B, a->Hkv, a->m, a->d, e, false, &v[2]) ||
        !bufs.add_view(a->out, a->B, a->Hq, a->n, a->d, e, true, &v[3]))
        return LARD_ERR_INVALID_ARG;
    if (!a->lse || !aligned(a->lse, 4) || (a->k_len && !aligned(a->k_len, 4))) return LARD_ERR_INVALID_ARG;
    const size_t need = cross_plan(*a).bytes();
    if (!workspace_ok(workspace, workspace_bytes, need)) return LARD_ERR_INVALID_ARG;
    bufs.add_flat(a->lse, static_cast<size_t>(a->B) * a->Hq * a->n * 4, true);
    bufs.add_flat(a->k_len, static_cast<size_t>(a->B) * 4, false);
    bufs.add_flat(workspace, need, true);
    if (!bufs.outputs_disjoint()) return LARD_ERR_INVALID_ARG;
    DeviceGuard guard;
    st = bufs.select_device();
    if (st != LARD_OK) return st;
    LARD_ATTN_DISPATCH(a->dtype, a->d, cross_fwd, *a, v, workspace, stream);
    return cudaGetLastError() == cudaSuccess ? LARD_OK : LARD_ERR_CUDA;
}

lard_status lard_cross_attn_bwd(const lard_cross_attn* a, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
    NvtxRange range("lard cross attention, gradients");
    lard_status st = cross_sizes(a);
    if (st != LARD_OK) return st;
    const int e = elem_bytes(a->dtype);
    Buffers bufs;
    lard_attn_view v[8];
    if (!bufs.add_view(a->q, a->B, a->Hq, a->n, a->d, e, false, &v[0]) ||
        !bufs.add_view(a->k, a->B, a->Hkv, a->m, a->d, e, false, &v[1]) ||
        !bufs.add_view(a->v, a->B, a->Hkv, a->m, a->d, e, false, &v[2]) ||
        !bufs.add_view(a->out, a->B, a->Hq, a->n, a->d, e, false, &v[3]) ||
        !bufs.add_view(a->dout, a->B, a->Hq, a->n, a->d, e, false, &v[4]) ||
        !bufs.add_view(a->dq, a->B, a->Hq, a->n, a->d, e, true, &v[5]) ||
        !bufs.add_view(a->dk, a->B, a->Hkv, a->m, a->d, e, true, &v[6]) ||
        !bufs.add_view(a->dv, a->B, a->Hkv, a->m, a->d, e, true, &v[7]))
        return LARD_ERR_INVALID_ARG;
    if (!a->lse || !aligned(a->lse, 4) || (a->k_len && !aligned(a->k_len, 4))) return LARD_ERR_INVALID_ARG;
    const size_t need = bwd_bytes(*a);
    if (!workspace_ok(workspace, workspace_bytes, need)) return LARD_ERR_INVALID_ARG;
    bufs.add_flat(a->lse, static_cast<size_t>(a->B) * a->Hq * a->n * 4, false);
    bufs.add_flat(a->k_len, static_cast<size_t>(a->B) * 4, false);
    bufs.add_flat(workspace, need, true);
    if (!bufs.outputs_disjoint()) return LARD_ERR_INVALID_ARG;
    DeviceGuard guard;
    st = bufs.select_device();
    if (st != LARD_OK) return st;
    LARD_ATTN_DISPATCH(a->dtype, a->d, cross_bwd, *a, v, workspace, stream);
    return cudaGetLastError() == cudaSuccess ? LARD_OK : LARD_ERR_CUDA;
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
    const size_t need = prefix_plan(*a).bytes();
    if (!workspace_ok(workspace, workspace_bytes, need)) return LARD_ERR_INVALID_ARG;
    bufs.add_flat(a->lse, static_cast<size_t>(a->B) * a->Hq * a->n * 4, true);
    if (a->S > 0) bufs.add_flat(a->s_len, static_cast<size_t>(a->B) * 4, false);
    bufs.add_flat(workspace, need, true);
    if (!bufs.outputs_disjoint()) return LARD_ERR_INVALID_ARG;
    DeviceGuard guard;
    st = bufs.select_device();
    if (st != LARD_OK) return st;
    LARD_ATTN_DISPATCH(a->dtype, a->d, prefix_fwd, *a, v, workspace, stream);
    return cudaGetLastError() == cudaSuccess ? LARD_OK : LARD_ERR_CUDA;
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
