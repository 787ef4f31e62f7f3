// mea_norm.cu -- normalisation of rows (the last axis): layer norm and rms
// norm, forward and backward.
//
//   forward    mean = sum x / C (0 for rms), invstd = 1 / sqrt(var + eps),
//              var = sum (x - mean)^2 / C, xhat = (x - mean) invstd,
//              y = gamma xhat + beta
//   backward   a = dy gamma, m1 = sum a / C (0 for rms), m2 = sum a xhat / C,
//              dx = invstd (a - m1 - xhat m2),
//              dgamma = sum over rows of dy xhat, dbeta = sum over rows of dy
//
// Both are bound by memory (8 to 14 operations per element).  A row is held
// in registers between its reduction and its output, so each tensor is read
// once: a group of threads owns a row, a power of two from 32 threads (whole
// reduction by shuffles) to a block.  The variance is a second pass over the
// registers (sum of (x - mean)^2), not a difference of two large sums.  Row
// sums are fp32: up to 32 terms in sequence in a thread, then a tree.
#include <cuda_runtime.h>

#include <cstdint>

#include "mea_device.cuh"
#include "mea_internal.h"
#include "mea_norm_api.h"
#include "mea_stream.cuh"

namespace mea {
namespace {

constexpr int kNormThreads = 256;      // threads of a block (more where one row needs more)
constexpr int kNormMaxThreads = 1024;
constexpr int kSlabRows = 1024;        // most rows whose terms one fp32 column sum takes
constexpr int kSlabs = 296;            // column-sum slabs of a large tensor (two per SM)
constexpr int kColX = 32, kColY = 8;   // threads of a column-sum block: columns x rows

// Column-sum slabs: a function of the row count only, so the order of the
// sums does not depend on the device.
inline int64_t norm_slabs(int64_t rows)
{
    int64_t s = (rows + kColY - 1) / kColY;
    if (s > kSlabs) s = kSlabs;
    const int64_t m = (rows + kSlabRows - 1) / kSlabRows;
    if (s < m) s = m;
    return s < 1 ? 1 : s;
}

// One element of a tensor that the kernel may also write (dx over x or dy).
template <typename T>
__device__ __forceinline__ float load1_rw(const void *p, int64_t i)
{
    if constexpr (Store<T>::kBytes == 2)
        return __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16);
    else
        return static_cast<const float *>(p)[i];
}

// VL parameters from item i (elements i VL ..), or `fill` where p is NULL.
template <typename TP, int VL>
__device__ __forceinline__ void load_params(const void *p, int64_t i, float fill, float (&f)[VL])
{
    if (!p) {
#pragma unroll
        for (int j = 0; j < VL; ++j) f[j] = fill;
    } else if constexpr (VL == 1) {
        f[0] = Store<TP>::load1(p, i);
    } else {
        constexpr int PV = Store<TP>::V;
        constexpr int n = VL < PV ? VL : PV;   // elements taken from each 16-byte vector (or half of one)
        if constexpr (VL < PV) {
            // four bf16 parameters beside four fp32 elements: 8 bytes
            const uint2 w = __ldg(static_cast<const uint2 *>(p) + i);
            f[0] = __uint_as_float(w.x << 16);
            f[1] = __uint_as_float(w.x & 0xffff0000u);
            f[2] = __uint_as_float(w.y << 16);
            f[3] = __uint_as_float(w.y & 0xffff0000u);
        } else {
#pragma unroll
            for (int q = 0; q < VL / n; ++q) {
                const uint4 w = __ldg(static_cast<const uint4 *>(p) + i * (VL / n) + q);
                float t[PV];
                Store<TP>::unpack(w, t);
#pragma unroll
                for (int j = 0; j < n; ++j) f[q * n + j] = t[j];
            }
        }
    }
}

// Sum over the group of 2^lg threads that owns a row, in every thread of the
// group.  Groups of more than a warp exchange through red (one float per
// warp), between two barriers that every thread of the block takes.
__device__ __forceinline__ float group_sum(float v, int lg, float *red)
{
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (lg > 5) {
        const int warp = threadIdx.x >> 5, wpg = 1 << (lg - 5), first = warp & ~(wpg - 1);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[warp] = v;
        __syncthreads();
        v = 0.f;
        for (int w = 0; w < wpg; ++w) v += red[first + w];
    }
    return v;
}

// ---------------------------------------------------------------- forward

template <typename T, typename TP, bool RMS, int VL, int NV>
__global__ void __launch_bounds__(kNormMaxThreads)
norm_fwd_kernel(const void *__restrict__ x, const void *__restrict__ gamma, const void *__restrict__ beta, float eps,
                void *__restrict__ y, float *__restrict__ mean_out, float *__restrict__ invstd_out, int64_t rows,
                int64_t C, int lg)
{
    using It = Item<T, VL>;
    __shared__ float red[32];
    const int g = threadIdx.x & ((1 << lg) - 1), G = 1 << lg;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> lg) + (threadIdx.x >> lg);
    const bool live = row < rows;
    const int items = (int)(C / VL);
    const int64_t base = row * items;
    const float rc = 1.f / (float)C;
    pdl_wait();
    typename It::Raw r[NV];
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (live && g + j * G < items) r[j] = It::load(x, base + g + j * G);
    float mean = 0.f;
    if constexpr (!RMS) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (live && g + j * G < items) {
                float f[VL];
                It::unpack(r[j], f);
                s += tree_sum(f);
            }
        mean = group_sum(s, lg, red) * rc;
    }
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (live && g + j * G < items) {
            float f[VL];
            It::unpack(r[j], f);
#pragma unroll
            for (int e = 0; e < VL; ++e) {
                f[e] -= mean;
                f[e] *= f[e];
            }
            q += tree_sum(f);
        }
    const float invstd = rsqrtf(fmaf(group_sum(q, lg, red), rc, eps));
    pdl_trigger();
    if (!live) return;
    if (g == 0) {
        if (!RMS && mean_out) mean_out[row] = mean;
        if (invstd_out) invstd_out[row] = invstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (g + j * G < items) {
            float f[VL], w[VL], b[VL];
            It::unpack(r[j], f);
            load_params<TP, VL>(gamma, g + j * G, 1.f, w);
            load_params<TP, VL>(beta, g + j * G, 0.f, b);
#pragma unroll
            for (int e = 0; e < VL; ++e) f[e] = fmaf((f[e] - mean) * invstd, w[e], b[e]);
            It::store(y, base + g + j * G, f);
        }
}

// Rows too long for the registers of a block: one block per row, which is
// read again for each of the passes.
template <typename T, typename TP, bool RMS>
__global__ void __launch_bounds__(kNormMaxThreads)
norm_fwd_long_kernel(const void *__restrict__ x, const void *__restrict__ gamma, const void *__restrict__ beta,
                     float eps, void *__restrict__ y, float *__restrict__ mean_out, float *__restrict__ invstd_out,
                     int64_t rows, int64_t C)
{
    __shared__ double red[32];
    __shared__ float bc;
    const int64_t row = blockIdx.x, base = row * C;
    pdl_wait();
    float mean = 0.f;
    if constexpr (!RMS) {
        double s = 0.0;
        for (int64_t i = threadIdx.x; i < C; i += blockDim.x) s += Store<T>::load1(x, base + i);
        s = block_sum(s, red);
        if (threadIdx.x == 0) bc = (float)(s / (double)C);
        __syncthreads();
        mean = bc;
        __syncthreads();
    }
    double q = 0.0;
    for (int64_t i = threadIdx.x; i < C; i += blockDim.x) {
        const float d = Store<T>::load1(x, base + i) - mean;
        q += (double)d * d;
    }
    q = block_sum(q, red);
    if (threadIdx.x == 0) bc = rsqrtf((float)(q / (double)C) + eps);
    __syncthreads();
    const float invstd = bc;
    pdl_trigger();
    if (threadIdx.x == 0) {
        if (!RMS && mean_out) mean_out[row] = mean;
        if (invstd_out) invstd_out[row] = invstd;
    }
    for (int64_t i = threadIdx.x; i < C; i += blockDim.x) {
        const float w = gamma ? Store<TP>::load1(gamma, i) : 1.f, b = beta ? Store<TP>::load1(beta, i) : 0.f;
        Store<T>::store1(y, base + i, fmaf((Store<T>::load1(x, base + i) - mean) * invstd, w, b));
    }
}

// --------------------------------------------------------------- backward

// Column sums of one slab of rows: partial[slab][0][c] = sum dy xhat,
// partial[slab][1][c] = sum dy.  A block covers 32 VL columns with 8 rows at
// a time; its 8 sums per column are added in order through shared memory.
template <typename T, bool RMS, int VL>
__global__ void __launch_bounds__(kColX *kColY)
norm_cols_kernel(const void *__restrict__ x, const void *__restrict__ dy, const float *__restrict__ mean,
                 const float *__restrict__ invstd, float *__restrict__ partial, int64_t rows, int64_t C,
                 int64_t per_slab, unsigned int col_blocks)
{
    using It = Item<T, VL>;
    __shared__ float red[kColY][kColX * VL * 2 + 1];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int items = (int)(C / VL);
    const unsigned int slab = blockIdx.x / col_blocks, col = blockIdx.x % col_blocks;
    const int64_t item = (int64_t)col * kColX + tx;
    const int64_t r0 = (int64_t)slab * per_slab, r1 = r0 + per_slab < rows ? r0 + per_slab : rows;
    float sg[VL] = {}, sb[VL] = {};
    pdl_wait();
    if (item < items) {
        for (int64_t r = r0 + ty; r < r1; r += kColY) {
            const float m = RMS ? 0.f : mean[r], is = invstd[r];
            float f[VL], d[VL];
            It::unpack(It::load(x, r * items + item), f);
            It::unpack(It::load(dy, r * items + item), d);
#pragma unroll
            for (int e = 0; e < VL; ++e) {
                sg[e] = fmaf(d[e], (f[e] - m) * is, sg[e]);
                sb[e] += d[e];
            }
        }
    }
    pdl_trigger();
#pragma unroll
    for (int e = 0; e < VL; ++e) {
        red[ty][tx * VL + e] = sg[e];
        red[ty][kColX * VL + tx * VL + e] = sb[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * kColX * VL; i += kColX * kColY) {
        const int half = i / (kColX * VL);
        const int64_t c = (int64_t)col * kColX * VL + i % (kColX * VL);
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kColY; ++k) s += red[k][i];
        if (c < C) partial[((int64_t)slab * 2 + half) * C + c] = s;
    }
}

// dgamma[c], dbeta[c]: the slabs' sums in order, in fp64.
template <typename TP>
__global__ void __launch_bounds__(kColX *kColY)
norm_finish_kernel(const float *__restrict__ partial, void *__restrict__ dgamma, void *__restrict__ dbeta, int64_t C,
                   int64_t slabs)
{
    __shared__ double red[kColY][kColX];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * kColX + tx;   // over 2 C: dgamma, then dbeta
    const bool beta = i >= C;
    void *out = beta ? dbeta : dgamma;
    const bool live = i < 2 * C && out;
    pdl_wait();
    double s = 0.0;
    if (live)
        for (int64_t k = ty; k < slabs; k += kColY) s += partial[k * 2 * C + i];
    red[ty][tx] = s;
    __syncthreads();
    pdl_trigger();
    if (ty == 0 && live) {
#pragma unroll
        for (int k = 1; k < kColY; ++k) s += red[k][tx];
        Store<TP>::store1(out, beta ? i - C : i, (float)s);
    }
}

// dx of one row per group of threads.  dx may be x or dy itself: every
// element is read before it is written, by the thread that writes it.
template <typename T, typename TP, bool RMS, int VL, int NV>
__global__ void __launch_bounds__(kNormMaxThreads)
norm_dx_kernel(const void *x, const void *dy, const void *__restrict__ gamma, const float *__restrict__ mean_in,
               const float *__restrict__ invstd_in, void *dx, int64_t rows, int64_t C, int lg)
{
    using It = Item<T, VL>;
    __shared__ float red[32];
    const int g = threadIdx.x & ((1 << lg) - 1), G = 1 << lg;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> lg) + (threadIdx.x >> lg);
    const bool live = row < rows;
    const int items = (int)(C / VL);
    const int64_t base = row * items;
    const float rc = 1.f / (float)C;
    pdl_wait();
    typename It::Raw rx[NV], rd[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (live && g + j * G < items) {
            rx[j] = It::load_rw(x, base + g + j * G);
            rd[j] = It::load_rw(dy, base + g + j * G);
        }
    const float mean = RMS || !live ? 0.f : mean_in[row], is = live ? invstd_in[row] : 0.f;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (live && g + j * G < items) {
            float f[VL], d[VL], w[VL];
            It::unpack(rx[j], f);
            It::unpack(rd[j], d);
            load_params<TP, VL>(gamma, g + j * G, 1.f, w);
#pragma unroll
            for (int e = 0; e < VL; ++e) {
                d[e] *= w[e];
                f[e] = d[e] * ((f[e] - mean) * is);
            }
            if (!RMS) s1 += tree_sum(d);
            s2 += tree_sum(f);
        }
    const float m1 = RMS ? 0.f : group_sum(s1, lg, red) * rc, m2 = group_sum(s2, lg, red) * rc;
    pdl_trigger();
    if (!live) return;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (g + j * G < items) {
            float f[VL], d[VL], w[VL];
            It::unpack(rx[j], f);
            It::unpack(rd[j], d);
            load_params<TP, VL>(gamma, g + j * G, 1.f, w);
#pragma unroll
            for (int e = 0; e < VL; ++e) f[e] = is * (fmaf(-((f[e] - mean) * is), m2, d[e] * w[e]) - m1);
            It::store(dx, base + g + j * G, f);
        }
}

template <typename T, typename TP, bool RMS>
__global__ void __launch_bounds__(kNormMaxThreads)
norm_dx_long_kernel(const void *x, const void *dy, const void *__restrict__ gamma, const float *__restrict__ mean_in,
                    const float *__restrict__ invstd_in, void *dx, int64_t rows, int64_t C)
{
    __shared__ double red[32];
    __shared__ float bc[2];
    const int64_t row = blockIdx.x, base = row * C;
    pdl_wait();
    const float mean = RMS ? 0.f : mean_in[row], is = invstd_in[row];
    double s1 = 0.0, s2 = 0.0;
    for (int64_t i = threadIdx.x; i < C; i += blockDim.x) {
        const float w = gamma ? Store<TP>::load1(gamma, i) : 1.f;
        const float a = load1_rw<T>(dy, base + i) * w;
        s1 += a;
        s2 += a * ((load1_rw<T>(x, base + i) - mean) * is);
    }
    s1 = block_sum(s1, red);
    s2 = block_sum(s2, red);
    if (threadIdx.x == 0) {
        bc[0] = RMS ? 0.f : (float)(s1 / (double)C);
        bc[1] = (float)(s2 / (double)C);
    }
    __syncthreads();
    pdl_trigger();
    for (int64_t i = threadIdx.x; i < C; i += blockDim.x) {
        const float w = gamma ? Store<TP>::load1(gamma, i) : 1.f;
        const float xh = (load1_rw<T>(x, base + i) - mean) * is;
        Store<T>::store1(dx, base + i, is * (fmaf(-xh, bc[1], load1_rw<T>(dy, base + i) * w) - bc[0]));
    }
}

// ------------------------------------------------------------ host side

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A row group's shape: 2^lg threads with nv items each; nv = 0 where a row
// does not fit the registers of a block.
struct Group {
    int lg, nv;
};
// The fewest threads that hold a row (a warp sums by shuffles alone and its
// loads are all in flight at once), but no fewer items in flight on the GPU
// than `rows` allows: with few rows a row is spread over more threads.
inline Group pick_group(int64_t items, int64_t rows, int nv_max)
{
    int nv_want = nv_max;
    while (nv_want > 1 && rows * ((items + nv_want - 1) / nv_want) < (int64_t)148 * 1024) nv_want >>= 1;
    int lg = 5;
    while (lg < 10 && ((int64_t)nv_want << lg) < items) ++lg;
    int nv = 1;
    while (((int64_t)nv << lg) < items) nv <<= 1;
    return Group{lg, nv <= nv_max ? nv : 0};
}

template <typename F>
cudaError_t by_nv(int nv, F f)
{
    switch (nv) {
    case 1: return f(std::integral_constant<int, 1>{});
    case 2: return f(std::integral_constant<int, 2>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 8: return f(std::integral_constant<int, 8>{});
    case 16: return f(std::integral_constant<int, 16>{});
    }
    return cudaErrorInvalidValue;
}

template <typename T, typename TP, bool RMS, int VL>
cudaError_t fwd_vl(const NormLaunch &a)
{
    const Group g = pick_group(a.C / VL, a.rows, 16);
    if (g.nv == 0)
        return launch_pdl(norm_fwd_long_kernel<T, TP, RMS>, dim3((unsigned)a.rows), dim3(kNormMaxThreads), 0, a.stream,
                          a.x, a.gamma, a.beta, a.eps, a.out, a.mean, a.invstd, a.rows, a.C);
    const int threads = (1 << g.lg) > kNormThreads ? (1 << g.lg) : kNormThreads;
    const int64_t per = threads >> g.lg;
    return by_nv(g.nv, [&](auto nv) {
        return launch_pdl(norm_fwd_kernel<T, TP, RMS, VL, decltype(nv)::value>,
                          dim3((unsigned)((a.rows + per - 1) / per)), dim3(threads), 0, a.stream, a.x, a.gamma, a.beta,
                          a.eps, a.out, a.mean, a.invstd, a.rows, a.C, g.lg);
    });
}

template <typename T, typename TP, bool RMS, int VL>
cudaError_t bwd_vl(const NormLaunch &a)
{
    if (a.dgamma || a.dbeta) {
        float *partial = static_cast<float *>(a.workspace);
        const int64_t slabs = norm_slabs(a.rows), per = (a.rows + slabs - 1) / slabs;
        const int64_t cb = (a.C + kColX * VL - 1) / (kColX * VL);
        cudaError_t e = launch_pdl(norm_cols_kernel<T, RMS, VL>, dim3((unsigned)(cb * slabs)),
                                   dim3(kColX * kColY), 0, a.stream, a.x, a.dy, a.mean_in, a.invstd_in, partial,
                                   a.rows, a.C, per, (unsigned)cb);
        if (e != cudaSuccess) return e;
        e = launch_pdl(norm_finish_kernel<TP>, dim3((unsigned)((2 * a.C + kColX - 1) / kColX)), dim3(kColX * kColY), 0,
                       a.stream, partial, a.dgamma, a.dbeta, a.C, slabs);
        if (e != cudaSuccess) return e;
    }
    const Group g = pick_group(a.C / VL, a.rows, 8);
    if (g.nv == 0)
        return launch_pdl(norm_dx_long_kernel<T, TP, RMS>, dim3((unsigned)a.rows), dim3(kNormMaxThreads), 0, a.stream,
                          a.x, a.dy, a.gamma, a.mean_in, a.invstd_in, a.out, a.rows, a.C);
    const int threads = (1 << g.lg) > kNormThreads ? (1 << g.lg) : kNormThreads;
    const int64_t per = threads >> g.lg;
    return by_nv(g.nv, [&](auto nv) -> cudaError_t {
        if constexpr (decltype(nv)::value > 8)
            return cudaErrorInvalidValue;
        else
            return launch_pdl(norm_dx_kernel<T, TP, RMS, VL, decltype(nv)::value>,
                              dim3((unsigned)((a.rows + per - 1) / per)), dim3(threads), 0, a.stream, a.x, a.dy,
                              a.gamma, a.mean_in, a.invstd_in, a.out, a.rows, a.C, g.lg);
    });
}

// Vector items where every row starts on a 16-byte boundary.
template <typename T, typename TP, bool RMS, bool BWD>
cudaError_t by_align(const NormLaunch &a)
{
    constexpr int V = Store<T>::V;
    const bool vec = a.C % V == 0 && aligned16(a.x) && aligned16(a.out) && aligned16(a.gamma) && aligned16(a.beta) &&
                     aligned16(a.dy);
    if constexpr (BWD)
        return vec ? bwd_vl<T, TP, RMS, V>(a) : bwd_vl<T, TP, RMS, 1>(a);
    else
        return vec ? fwd_vl<T, TP, RMS, V>(a) : fwd_vl<T, TP, RMS, 1>(a);
}

template <typename T, typename TP, bool BWD>
cudaError_t by_norm(const NormLaunch &a)
{
    return a.rms ? by_align<T, TP, true, BWD>(a) : by_align<T, TP, false, BWD>(a);
}

template <bool BWD>
cudaError_t by_type(const NormLaunch &a)
{
    if (a.dtype == kBF16) return a.pdtype == kBF16 ? by_norm<Bf16, Bf16, BWD>(a) : by_norm<Bf16, float, BWD>(a);
    return a.pdtype == kBF16 ? by_norm<float, Bf16, BWD>(a) : by_norm<float, float, BWD>(a);
}

}  // namespace

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t C)
{
    if (rows <= 0 || C <= 0) return 0;
    return (size_t)norm_slabs(rows) * 2 * (size_t)C * sizeof(float);
}

cudaError_t launch_norm_fwd(const NormLaunch &a) { return by_type<false>(a); }
cudaError_t launch_norm_bwd(const NormLaunch &a) { return by_type<true>(a); }

}  // namespace mea
